"""Measured cases of the paged key/value cache operators.

Four operators of a serving loop that keeps its keys and values in pages:

* ``write``  -- new tokens' keys and values go into the pages of their sequences,
  as they are (bf16) or in 8 bits with one power-of-two scale per row and head;
* ``read``   -- the rows of every sequence come back from their pages, packed, in bf16;
* ``chunk``  -- attention of a chunk of new tokens per sequence over all of its
  cached keys, the chunk's own among them (causal);
* ``decode`` -- the same for one new token per sequence over an 8 bit cache.

The 8 bit form of a row x (one token, one head): with a the largest magnitude of
its finite values, e is the smallest whole number in [-60, 60] with
a <= 448 * 2^e; the codes are the e4m3 values nearest x * 2^-e (ties to even,
magnitudes over 448 to 448, infinities and NaN to NaN) and the scale byte is
e + 127.  A code c stands for c * 2^e.

A case gives sizes; ``lens`` seeds the lengths of its sequences, so that they
belong to the case and not to the inputs' seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
E_MIN, E_MAX, E_BIAS = -60, 60, 127
DEV = "cuda"


# ---------------------------------------------------------------------------- the cases


def _case(name, op, d, hq, hkv, page, b, new, past, q8, lens=1):
    """new, past: "lo-hi" ranges of new tokens and of keys cached before them, per sequence."""
    return {"name": name, "op": op, "d": d, "hq": hq, "hkv": hkv, "page": page, "b": b, "new": new, "past": past,
            "q8": q8, "lens": lens}


def listed():
    return [
        # one serving step of a batch of 64 requests writes one token each: latency
        _case("write 64 tokens 8 bit", "write", 128, 32, 32, 16, 64, "1-1", "511-16383", True),
        # an 8192 token prompt goes into the cache
        _case("write 8192 tokens 8 bit", "write", 128, 32, 32, 16, 1, "8192-8192", "0-0", True),
        # prompts of different lengths into a bf16 cache of small heads, pages that are no power of two
        _case("write ragged bf16 d64", "write", 64, 16, 16, 24, 16, "1-1024", "0-500", False),
        # one short sequence leaves the cache (moved, or handed to a dense call)
        _case("read 1000 keys 8 bit d64", "read", 64, 16, 16, 16, 1, "0-0", "1000-1000", True),
        # a batch of sequences leaves the cache
        _case("read 16 sequences 8 bit", "read", 128, 32, 8, 16, 16, "0-0", "512-16384", True),
        # four drafted tokens a request, to be verified in one pass over the batch
        _case("chunk 4 tokens x 64 8 bit", "chunk", 128, 32, 8, 16, 64, "4-4", "508-16380", True),
        # a 512 token piece of a long prompt over what is cached of it
        _case("chunk 512 over 16K 8 bit", "chunk", 128, 32, 8, 64, 1, "512-512", "15872-15872", True),
        # an 8192 token prompt in one piece, one key head per query head
        _case("chunk 8192 bf16", "chunk", 128, 32, 32, 16, 1, "8192-8192", "0-0", False),
        # a mixed step: single tokens beside prompts' pieces, small heads
        _case("chunk ragged bf16 d64", "chunk", 64, 16, 16, 24, 16, "1-700", "0-4096", False),
        # the smallest call: one request at its beginning
        _case("decode 100 keys 8 bit", "decode", 128, 32, 32, 16, 1, "1-1", "99-99", True),
        # one request of 8192 keys
        _case("decode 8192 keys 8 bit", "decode", 128, 32, 32, 16, 1, "1-1", "8191-8191", True),
        # the 64 request batch, four query heads to a key head
        _case("decode 64 requests 8 bit", "decode", 128, 32, 8, 16, 64, "1-1", "511-16383", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: an operator, its head layout and types, and lengths over the logarithm of their range,
    within the largest listed case's data (131072 cached rows of eight 128-wide heads) and products."""
    op = rng.choice(["write", "read", "chunk", "chunk", "decode"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    hq = hkv * group if hkv * group <= 64 else hkv
    page = rng.choice([8, 16, 24, 32, 48, 64, 128, 256])
    b = _log(rng, 1, 64)
    rows = 131072 * 8 * 128 // (hkv * d)  # cached rows that are allowed in all
    past = max(1, min(_log(rng, 1, 16384), rows // (2 * b)))
    lo = rng.choice([past, max(1, past // 8), 0])
    q8 = True if op == "decode" else rng.random() < 0.6
    if op == "read":
        new = "0-0"
    elif op == "decode":
        new = "1-1"
    else:
        most = max(1, min(_log(rng, 1, 8192), rows // (4 * b)))
        if op == "chunk":  # 4 d hq pairs: at most half of the 8192 token prompt's
            most = max(1, min(most, 8192 * 8192 * 32 * 128 // 4 // (d * hq * b * (past + most))))
        new = "%d-%d" % (rng.choice([most, 1]), most)
    return {"op": op, "d": d, "hq": hq, "hkv": hkv, "page": page, "b": b, "new": new, "past": "%d-%d" % (lo, past),
            "q8": q8, "lens": rng.randrange(1 << 30)}


def _lengths(case):
    """New tokens and all keys (the new ones among them) of every sequence."""
    r = random.Random(case["lens"])
    n0, n1 = (int(x) for x in case["new"].split("-"))
    p0, p1 = (int(x) for x in case["past"].split("-"))
    new = [r.randint(n0, n1) for _ in range(case["b"])]
    return new, [n + r.randint(p0, p1) for n in new]


# ---------------------------------------------------------------------------- inputs


def _offsets(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _to_8bit(x):
    """The codes (e4m3) and scale bytes of rows x [..., d]."""
    x = x.float()
    good = torch.isfinite(x)
    a = torch.where(good, x, 0.0).abs().amax(-1)
    f, e = torch.frexp(a)  # a = f 2^e, f in [1/2, 1): a <= 448 2^k = (7/8) 2^(k + 9)
    k = torch.where(f <= 0.875, e - 9, e - 8)
    k = torch.where(a == 0, torch.full_like(k, E_MIN), k).clamp(E_MIN, E_MAX)
    y = torch.ldexp(x, -k[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    y = torch.where(good, y, float("nan"))
    return y.to(torch.float8_e4m3fn), (k + E_BIAS).to(torch.uint8)


def _rows(shape, gen):
    """Keys or values as projections give them: heads of different loudness, a few loud channels."""
    x = torch.randn(shape, generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn(shape[-2:-1] + (1,), generator=gen, device=DEV))
    x *= 1.0 + 3.0 * (torch.rand((1,) + shape[-1:], generator=gen, device=DEV) < 0.03)
    return x.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    new, keys = _lengths(case)
    b, hq, hkv, d, page = (case[k] for k in ("b", "hq", "hkv", "d", "page"))
    per = [-(-n // page) for n in keys]
    pages = max(1, sum(per)) + 3  # three that belong to no sequence
    order = torch.randperm(pages, generator=gen, device=DEV).cpu().tolist()
    table, at = [], 0
    for n in per:
        table.append(order[at:at + n] + [-1] * (max(1, max(per)) - n))
        at += n
    s = {"case": dict(case), "new": new, "keys": keys,
         "table": torch.tensor(table, dtype=torch.int32, device=DEV), "cu_new": _offsets(new), "cu_keys": _offsets(keys),
         "seqlens": torch.tensor(keys, dtype=torch.int32, device=DEV), "k_scales": None, "v_scales": None}
    for name in ("k", "v"):
        if case["op"] == "write":  # an empty cache and the rows to go into it
            s[name + "_new"] = _rows((sum(new), hkv, d), gen)
            s[name + "_pages"] = torch.zeros((pages, page, hkv, d), device=DEV, dtype=torch.bfloat16)
            if case["q8"]:
                s[name + "_pages"] = s[name + "_pages"].to(torch.float8_e4m3fn)
                s[name + "_scales"] = torch.full((pages, page, hkv), E_BIAS, dtype=torch.uint8, device=DEV)
        else:
            s[name + "_pages"] = _rows((pages, page, hkv, d), gen)
            if case["q8"]:
                s[name + "_pages"], s[name + "_scales"] = _to_8bit(s[name + "_pages"])
    if case["op"] in ("chunk", "decode"):
        s["q"] = torch.randn((sum(new), hq, d), generator=gen, device=DEV).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------- the plain forms


def _slots(s, pos, seq):
    """Row of the flattened pages that holds key `pos` of sequence `seq` (page 0 where the table has none)."""
    page = s["case"]["page"]
    at = torch.div(pos, page, rounding_mode="floor").clamp(max=s["table"].shape[1] - 1)
    return s["table"][seq, at].long().clamp(min=0) * page + pos % page


def _sequence_of(cu, total):
    """Sequence and place in it of each of `total` packed rows."""
    row = torch.arange(total, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return seq, row - cu[seq]


def _values(s, name, slots):
    """The cache's rows at `slots`, in 32 bits."""
    x = s[name + "_pages"].flatten(0, 1)[slots].float()
    if s[name + "_scales"] is not None:
        x = torch.ldexp(x, (s[name + "_scales"].flatten(0, 1)[slots].int() - E_BIAS)[..., None])
    return x


def _write(s):
    seq, i = _sequence_of(s["cu_new"], sum(s["new"]))
    pos = s["seqlens"][seq] - (s["cu_new"][seq + 1] - s["cu_new"][seq]) + i
    slots = _slots(s, pos, seq)
    out = {}
    for name in ("k", "v"):
        rows, pages = s[name + "_new"], s[name + "_pages"].flatten(0, 1)
        if s["case"]["q8"]:
            rows, scales = _to_8bit(rows)
            s[name + "_scales"].flatten(0, 1)[slots] = scales
            out[name + "_scales"] = s[name + "_scales"]
            pages.view(torch.uint8)[slots] = rows.view(torch.uint8)
        else:
            pages[slots] = rows
        out[name] = s[name + "_pages"]
    return out


def _read(s):
    seq, i = _sequence_of(s["cu_keys"], sum(s["keys"]))
    slots = _slots(s, i, seq)
    return {name: _values(s, name, slots).to(torch.bfloat16) for name in ("k", "v")}


def _attend(s):
    c = s["case"]
    b, hq, hkv, d = c["b"], c["hq"], c["hkv"], c["d"]
    n, m = max(s["new"]), max(s["keys"])
    seq, i = _sequence_of(s["cu_new"], sum(s["new"]))
    q = torch.zeros((b, n, hq, d), device=DEV)
    q[seq, i] = s["q"].float()
    q = q.view(b, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)  # rows: token, head of the group
    every = torch.arange(b, device=DEV)[:, None]
    slots = _slots(s, torch.arange(m, device=DEV)[None].expand(b, m), every)
    x = (q @ _values(s, "k", slots).permute(0, 2, 3, 1)) / math.sqrt(d)
    new = s["cu_new"].diff()[:, None]
    last = s["seqlens"][:, None] - new + torch.arange(n, device=DEV)[None]  # the last key that each token sees
    seen = torch.arange(m, device=DEV)[None, None] <= torch.minimum(last, s["seqlens"][:, None] - 1)[..., None]
    seen = seen.repeat_interleave(hq // hkv, 1)[:, None]
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ _values(s, "v", slots).permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).view(b, hkv, n, hq // hkv).permute(0, 1, 3, 2).reshape(b, hq, n)
    o = o.view(b, hkv, n, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, n, hq, d)[seq, i].to(torch.bfloat16)
    if c["op"] == "decode":
        return {"o": o, "lse": lse[..., 0]}
    return {"o": o, "lse": lse.transpose(0, 1)[:, seq, i]}


def run(s):
    c = s["case"]
    if not own:
        return {"write": _write, "read": _read, "chunk": _attend, "decode": _attend}[c["op"]](s)
    import exact_io_aware_54_b200 as fa
    if c["op"] == "write":
        fa.fa_cache_write(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["cu_new"], s["table"], s["seqlens"],
                          k_scales=s["k_scales"], v_scales=s["v_scales"])
        out = {"k": s["k_pages"], "v": s["v_pages"]}
        return out | {"k_scales": s["k_scales"], "v_scales": s["v_scales"]} if c["q8"] else out
    if c["op"] == "read":
        k, v = fa.fa_cache_read(s["k_pages"], s["v_pages"], s["cu_keys"], s["table"], sum(s["keys"]),
                                k_scales=s["k_scales"], v_scales=s["v_scales"])
        return {"k": k, "v": v}
    if c["op"] == "chunk":
        o, lse = fa.fa_fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["cu_new"], s["table"], s["seqlens"],
                                 max(s["new"]), max(s["keys"]), causal=True, k_scales=s["k_scales"],
                                 v_scales=s["v_scales"])
    else:
        o, lse = fa.fa_decode_paged_q8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"],
                                       s["seqlens"], max(s["keys"]))
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    new, keys = _lengths(case)
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["b"]
    row = hkv * (d + 1 if case["q8"] else 2 * d)  # one token's keys or values in the cache
    index = 4 * (2 * b + sum(-(-n // case["page"]) for n in keys))
    if case["op"] == "write":
        return {"bytes": 2 * sum(new) * (2 * hkv * d + row) + index, "flops": 4 * sum(new) * hkv * d}
    if case["op"] == "read":
        return {"bytes": 2 * sum(keys) * (2 * hkv * d + row) + index, "flops": 2 * sum(keys) * hkv * d}
    used = [k for n, k in zip(new, keys) if n]
    pairs = sum(n * k - n * (n - 1) // 2 for n, k in zip(new, keys))
    return {"bytes": 2 * sum(used) * row + sum(new) * hq * (4 * d + 4) + index, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------- the definition in 64 bits


def _exact_rows(s, name, b):
    """Keys or values of sequence b, page by page, in 64 bits: [keys, hkv, d]."""
    c, n = s["case"], s["keys"][b]
    ids = s["table"][b, : -(-n // c["page"])].long()
    x = s[name + "_pages"][ids].double()
    if s[name + "_scales"] is not None:
        x = x * torch.pow(2.0, s[name + "_scales"][ids].double() - 127.0)[..., None]
    return x.flatten(0, 1)[:n]


def _exact_8bit(x):
    """Nearest codes by a search of the table of all e4m3 values, in 64 bits."""
    x = x.double()
    bad = ~torch.isfinite(x)
    a = x.masked_fill(bad, 0.0).abs().amax(-1)
    scale = torch.full_like(a, 2.0 ** E_MIN)
    for e in range(E_MIN, E_MAX):
        scale = torch.where(a > E4M3_MAX * 2.0 ** e, 2.0 ** (e + 1), scale)
    # code m (0 .. 126) stands for (8 + m % 8) 2^(m // 8 - 10) from m = 8 on, for m 2^-9 below
    mags = [m * 2.0 ** -9 if m < 8 else (8 + m % 8) * 2.0 ** (m // 8 - 10) for m in range(127)]
    table = torch.tensor(mags, dtype=torch.float64, device=DEV)
    y = (x.masked_fill(bad, 0.0) / scale[..., None]).abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(table, y.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - y, y - table[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (table[code] * torch.sign(x.masked_fill(bad, 0.0))).masked_fill(bad, math.nan), torch.log2(scale)


def exact(case, seed):
    new, keys = _lengths(case)
    if case["op"] in ("chunk", "decode") and 4 * case["d"] * case["hq"] * sum(n * k for n, k in zip(new, keys)) > 3e12:
        return None
    s = prepare(case, seed)
    c = s["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    if c["op"] == "write":
        out = {}
        for name in ("k", "v"):
            pages = s[name + "_pages"].double()
            scales = None if s[name + "_scales"] is None else s[name + "_scales"].long()
            at = 0
            for b, (n, total) in enumerate(zip(new, keys)):
                pos = torch.arange(total - n, total, device=DEV)
                rows = s[name + "_new"][at:at + n]
                ids = s["table"][b].long()[pos // page]
                if scales is not None:
                    rows, e = _exact_8bit(rows)
                    scales[ids, pos % page] = e.round().long() + 127
                pages[ids, pos % page] = rows.double()
                at += n
            out[name] = pages
            if scales is not None:
                out[name + "_scales"] = scales
        return out
    if c["op"] == "read":
        return {name: torch.cat([_exact_rows(s, name, b) for b in range(c["b"])]) for name in ("k", "v")}
    o, lse, at = [], [], 0
    for b, (n, total) in enumerate(zip(new, keys)):
        q = s["q"][at:at + n].double()
        k, v = _exact_rows(s, "k", b), _exact_rows(s, "v", b)
        at += n
        ob, lb = torch.zeros((n, hq, d), dtype=torch.float64, device=DEV), torch.zeros((hq, n), dtype=torch.float64, device=DEV)
        hidden = torch.ones((n, total), dtype=torch.bool, device=DEV).triu(total - n + 1)
        for h in range(hq):
            x = torch.matmul(q[:, h], k[:, h * hkv // hq].T) * d ** -0.5
            x = x.masked_fill(hidden, -math.inf)
            lb[h] = torch.logsumexp(x, -1)
            ob[:, h] = torch.nan_to_num(torch.exp(x - lb[h][:, None]), nan=0.0) @ v[:, h * hkv // hq]
        o.append(ob)
        lse.append(lb)
    lse = torch.cat(lse, 1)
    return {"o": torch.cat(o), "lse": lse.T if c["op"] == "decode" else lse}
