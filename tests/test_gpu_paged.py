"""GPU parity of the paged cache operators: writing and reading a cache (bf16, 8 bit),
attention of new tokens over it, single tokens over the 8 bit one."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_54_b200 as fa
from exact_io_aware_54_b200 import synth
from oracle import paged
from tests._harness import f64

pytestmark = pytest.mark.gpu

INVALID = 1


def _check(expect=0):
    assert fa.fa_check(fa.paged_workspace()) == expect


class Cache:
    """A paged cache of random rows: pages scattered, three to spare, rows that belong to
    no sequence filled with `junk`."""

    def __init__(self, seed, lens, H, d, page, q8, spread=0.0, junk=None):
        self.lens, self.q8, self.H, self.d, self.page = list(lens), q8, H, d, page
        _, k, v, table, seqlens = synth.paged_decode_inputs(seed, lens, H, d, page)
        rng = np.random.default_rng(seed)
        loud = torch.from_numpy(np.exp2(rng.uniform(-spread, spread, k.shape[:3] + (1,)))) if spread else 1.0
        self.values, self.pages, self.scales = {}, {}, {}
        used = torch.zeros(k.shape[:2], dtype=torch.bool)
        for b, n in enumerate(self.lens):
            t = torch.arange(n)
            used[table[b, t // page].long(), t % page] = True
        for name, x in (("k", k), ("v", v)):
            x = (x.double() * loud).to(torch.bfloat16) if name == "v" else x
            if q8:
                codes, scales = paged.quantise(f64(x))
                self.values[name] = paged.dequantise(codes, scales)
                codes, scales = torch.from_numpy(codes), torch.from_numpy(scales)
                if junk is not None:
                    codes[~used] = 0x7F
                    scales[~used] = 255
                self.scales[name] = scales.cuda()
                self.pages[name] = codes.view(torch.float8_e4m3fn).cuda()
            else:
                self.values[name] = f64(x)
                if junk is not None:
                    x[~used] = junk
                self.pages[name] = x.cuda()
        self.table, self.seqlens = table.cuda(), seqlens.cuda()

    @property
    def kw(self):
        return dict(k_scales=self.scales["k"], v_scales=self.scales["v"]) if self.q8 else {}

    def reference(self, b, q, causal):
        n = self.lens[b]
        row = self.table[b].cpu().numpy()
        k, v = (paged.gather(self.values[x], row, n) for x in "kv")
        vs = np.exp2(paged.gather(f64(self.scales["v"]), row, n) - 127.0) if self.q8 else None
        return paged.attend(q, k, v, causal, 1 / math.sqrt(self.d), vs)


def _close(o, lse, ref, what):
    """o [n, Hq, d], lse [n, Hq] against (o, lse, o_tol, lse_tol)."""
    ro, rl, to, tl = ref
    o, lse = f64(o), f64(lse)
    assert np.isfinite(o).all(), what
    assert (np.abs(o - ro) <= to).all(), f"{what}: o off by {(np.abs(o - ro) / to).max():.2f} tolerances"
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), none), what
    d = np.where(none, 0.0, np.abs(np.where(none, 0, lse) - np.where(none, 0, rl)))
    assert (d <= tl).all(), f"{what}: lse off by {(d / tl).max():.2f} tolerances"


def _decode(c, hq, seed, max_k=None, **kw):
    q = synth._normal((len(c.lens), hq, c.d), seed)
    o, lse = fa.fa_decode_paged_q8(q.cuda(), c.pages["k"], c.pages["v"], c.scales["k"], c.scales["v"], c.table,
                                   c.seqlens, max(c.lens) if max_k is None else max_k, **kw)
    _check()
    for b in range(len(c.lens)):
        _close(o[b:b + 1], lse[b:b + 1], c.reference(b, f64(q[b:b + 1]), True), f"sequence {b}, {c.lens[b]} keys")
    return q, o, lse


def _chunk(c, hq, new, seed, causal=True, pad=0, q=None):
    cu = synth.cu_seqlens_of(new).cuda()
    total = int(sum(new)) + pad
    q = synth._normal((total, hq, c.d), seed) if q is None else q
    o = torch.full((total, hq, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq, total), 7.0, device="cuda")
    fa.fa_fwd_paged(q.cuda(), c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, max(new), max(max(c.lens), 0), causal,
                    out=o, lse=lse, **c.kw)
    _check()
    at = 0
    for b, n in enumerate(new):
        _close(o[at:at + n], lse[:, at:at + n].T, c.reference(b, f64(q[at:at + n]), causal),
               f"sequence {b}, {n} over {c.lens[b]}")
        at += n
    if pad:
        assert (o[at:] == 7).all() and (lse[:, at:] == 7).all(), "rows behind the last sequence were written"
    return o, lse


# ------------------------------------------------------------------------------- single tokens

LENS = [1, 7, 0, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 128, 384])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_pages(d, page):
    _decode(Cache(10 + page, LENS, 2, d, page, True), 4, 20 + page)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (5, 1), (12, 3), (24, 1), (40, 1), (32, 8), (130, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_heads(d, hq, hkv):
    """Head layouts through every row tile: groups of 1 to 65, odd key heads."""
    _decode(Cache(hq, [5, 513], hkv, d, 16, True), hq, 30 + hq)


def test_decode_long_and_short():
    """Stretches of many CTAs and many sequences in one CTA."""
    _decode(Cache(40, [16384], 1, 128, 64, True), 4, 41)
    _decode(Cache(42, [i % 9 for i in range(700)], 1, 64, 8, True), 1, 43)


def test_decode_value_scales():
    """Values whose scales differ by up to 2^20 between keys and heads."""
    _decode(Cache(44, [1, 50, 700], 3, 128, 16, True, spread=10.0), 6, 45)
    _decode(Cache(44, [1, 50, 700], 3, 64, 16, True, spread=10.0), 6, 45)


def test_decode_loud_queries():
    """Scores over a range of hundreds: the running maximum moves, nearly one-hot rows."""
    c = Cache(46, [900, 1300], 2, 128, 16, True)
    q = synth._normal((2, 8, 128), 47, mult=40.0)
    o, lse = fa.fa_decode_paged_q8(q.cuda(), c.pages["k"], c.pages["v"], c.scales["k"], c.scales["v"], c.table, c.seqlens,
                                   1300)
    _check()
    for b in range(2):
        _close(o[b:b + 1], lse[b:b + 1], c.reference(b, f64(q[b:b + 1]), True), f"sequence {b}")


# ------------------------------------------------------------------------------- chunks


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [3, 16, 48, 256])
def test_chunk_mixed(d, q8, causal, page):
    """Single tokens, no tokens, and chunks that cross row tiles, one pass; rows behind."""
    new = [1, 0, 3, 17, 70, 130, 1]
    lens = [1, 40, 3, 500, 71, 300, 1000]
    _chunk(Cache(50 + page, lens, 2, d, page, q8, junk=math.nan), 4, new, 60 + page, causal, pad=5)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 2), (7, 1), (15, 5), (64, 2), (96, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_heads(d, hq, hkv, q8):
    _chunk(Cache(70 + hq, [33, 200], hkv, d, 16, q8), hq, [5, 40], 80 + hq)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [127, 128, 129, 255, 256, 257, 700])
def test_chunk_lengths(d, q8, n):
    """A chunk from empty, and over some keys, around the tiles' edges."""
    _chunk(Cache(90 + n, [n, n + 131], 2, d, 32, q8, junk=math.inf), 4, [n, n], 91 + n)


@pytest.mark.parametrize("q8", [False, True])
def test_chunk_rows_that_see_nothing(q8):
    """More tokens than keys (the first see none), and no keys at all."""
    for n in (9, 300):
        c = Cache(100, [4, 0, 130], 2, 128, 16, q8, junk=math.nan)
        _chunk(c, 4, [n, n, n], 101)
        _chunk(c, 4, [n, n, n], 102, causal=False)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_loud(d, q8):
    c = Cache(110, [400, 900], 2, d, 16, q8)
    q = synth._normal((2 + 300, 4, d), 111, mult=40.0)
    _chunk(c, 4, [2, 300], 0, q=q)


@pytest.mark.parametrize("q8", [False, True])
def test_chunk_long_context(q8):
    """Few rows over a long cache (many CTAs share one problem), and more rows than a tile."""
    c = Cache(120, [9000], 1, 128, 64, q8)
    _chunk(c, 8, [4], 121)
    _chunk(c, 8, [100], 122)


@pytest.mark.parametrize("power", [-66, 55])
@pytest.mark.parametrize("n", [3, 200])
def test_chunk_scale_ends(n, power):
    """Values at the ends of the 8 bit format's scales (codes below the normal numbers at
    the lower end), keys as quiet as that beside them."""
    c = Cache(125, [n + 70], 2, 128, 16, True)
    rng = np.random.default_rng(126)
    for name, shift in (("k", -66 if power < 0 else 0), ("v", power)):
        x = torch.from_numpy(rng.standard_normal(c.values[name].shape) * 2.0 ** shift).to(torch.bfloat16)
        codes, scales = paged.quantise(f64(x))
        c.values[name] = paged.dequantise(codes, scales)
        c.pages[name] = torch.from_numpy(codes).view(torch.float8_e4m3fn).cuda()
        c.scales[name] = torch.from_numpy(scales).cuda()
    _chunk(c, 4, [n], 127)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n", [1, 150])
def test_chunk_not_finite(n, q8, d):
    """A NaN in the cache comes out as one: of a key, in every token that sees it; of a value, in its dims."""
    L, at, head = 300, 20, 1
    c = Cache(150, [L], 2, d, 16, q8)
    page, row = int(c.table[0, at // 16]), at % 16
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q = synth._normal((n, 4, d), 151).cuda()
    call = lambda: fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, n, L, True, **c.kw)
    good, _ = call()
    mine = torch.arange(4, device="cuda") // 2 == head
    for name, dims in (("v", [0, 5, 17, d - 1]), ("k", [d // 2 + 3])):
        pages = c.pages[name].view(torch.uint8) if q8 else c.pages[name]
        old = pages.clone()
        for i in dims:
            pages[page, row, head, i] = (0x7F if i % 2 else 0xFF) if q8 else math.nan
        o, lse = call()
        _check()
        pages.copy_(old)
        if name == "k":
            assert o[:, mine].isnan().all() and lse[mine].isnan().all()
            if d == 128:
                assert torch.equal(o[:, ~mine], good[:, ~mine])
        else:
            hit = torch.zeros(d, dtype=torch.bool, device="cuda")
            hit[dims] = True
            assert o[:, mine][..., hit].isnan().all()
            assert torch.equal(o[:, mine][..., ~hit], good[:, mine][..., ~hit])
            assert torch.equal(o[:, ~mine], good[:, ~mine])


def test_workspace_is_the_streams():
    """A bad page is recorded where fa_check looks on that stream, and nowhere else."""
    c = Cache(128, [40], 1, 64, 16, True)
    q = synth._normal((1, 1, 64), 129).cuda()
    table = torch.full_like(c.table, -1)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        fa.fa_decode_paged_q8(q, c.pages["k"], c.pages["v"], c.scales["k"], c.scales["v"], table, c.seqlens, 40)
    torch.cuda.synchronize()
    _check()
    with torch.cuda.stream(other):
        _check(INVALID)
    ws = torch.zeros(fa.fa_paged_workspace_size(1, 1, 1, 1, 40, 64), dtype=torch.uint8, device="cuda")
    fa.fa_decode_paged_q8(q, c.pages["k"], c.pages["v"], c.scales["k"], c.scales["v"], table, c.seqlens, 40, ws=ws)
    assert fa.fa_check(ws) == INVALID
    _check()


def test_binding_refusals():
    c = Cache(132, [40], 2, 64, 16, True)
    q = synth._normal((1, 2, 64), 133).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    args = dict(k_pages=c.pages["k"], v_pages=c.pages["v"], block_table=c.table, seqlens_k=c.seqlens, max_seqlen_k=40,
                **c.kw)
    fwd = dict(q=q, cu_seqlens_q=cu, max_seqlen_q=1)
    for bad in (dict(q=q.float()), dict(q=q.expand(1, 2, 64).transpose(1, 2)), dict(k_pages=c.pages["k"][:, :, :1]),
                dict(k_scales=None), dict(k_scales=c.scales["k"].int()), dict(k_scales=c.scales["k"][:1]),
                dict(block_table=c.table.long()), dict(block_table=c.table[0]), dict(seqlens_k=c.seqlens.cpu()),
                dict(cu_seqlens_q=cu.long()), dict(cu_seqlens_q=cu[None]), dict(k_pages=c.pages["k"].view(torch.uint8)),
                dict(out=torch.empty(1, 2, 64, device="cuda")), dict(lse=torch.empty(1, 2, device="cuda")),
                dict(ws=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            fa.fa_fwd_paged(**{**args, **fwd, **bad})
    for bad in (dict(max_seqlen_k=1 << 20), dict(ws=torch.zeros(64, dtype=torch.uint8, device="cuda")), dict(max_seqlen_q=0)):
        with pytest.raises(fa.FAError):
            fa.fa_fwd_paged(**{**args, **fwd, **bad})
    with pytest.raises(ValueError):  # a bf16 cache where the pages are 8 bit
        fa.fa_fwd_paged(**{**args, **fwd, "k_scales": None, "v_scales": None})
    with pytest.raises(ValueError):
        fa.fa_decode_paged_q8(**{**args, "q": q, "k_scales": None})
    x = synth._normal((1, 2, 64), 134).cuda()
    write = dict(k=x, v=x, cu_seqlens=cu, **{k: v for k, v in args.items() if k != "max_seqlen_k"})
    for bad in (dict(k=x.float()), dict(v=x[:, :1]), dict(k=x.cpu()), dict(cu_seqlens=cu[:1]), dict(v_scales=None)):
        with pytest.raises(ValueError):
            fa.fa_cache_write(**{**write, **bad})
    _check()


@pytest.mark.parametrize("n", [2, 200])
def test_chunk_strided_queries(n):
    """q as a slice of a fused projection."""
    c = Cache(130, [n + 60], 2, 128, 16, True)
    wide = synth._normal((n, 4 + 2 + 2, 128), 131).cuda()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    args = (c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, n, n + 60, True)
    o, lse = fa.fa_fwd_paged(wide[:, 2:6], *args, **c.kw)
    o2, lse2 = fa.fa_fwd_paged(wide[:, 2:6].contiguous(), *args, **c.kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q8", [False, True])
def test_chunk_agrees_with_packed_forward(q8):
    """The same keys read back and given to the packed forward."""
    c = Cache(140, [150, 40, 513], 4, 128, 16, q8)
    new = [150, 7, 200]
    q = synth._normal((sum(new), 4, 128), 141)
    o, lse = _chunk(c, 4, new, 0, q=q)
    cu = synth.cu_seqlens_of(c.lens).cuda()
    k, v = fa.fa_cache_read(c.pages["k"], c.pages["v"], cu, c.table, sum(c.lens), **c.kw)
    o2, lse2 = fa.fa_fwd_varlen(q.cuda(), k, v, synth.cu_seqlens_of(new).cuda(), cu, 200, 513, causal=True)
    assert (lse - lse2).abs().max() <= 1e-4 * 10
    # two roundings of o and of the weights: 4 half steps of 2^-8
    assert ((o.double() - o2.double()).abs() <= 4 * 2.0 ** -8 * 4.0).all()


def test_repeatable():
    """No atomics: the same call gives the same bits."""
    c = Cache(150, [5000, 30, 700], 2, 128, 16, True)
    for new in ([1, 1, 1], [4, 2, 500]):
        a = _chunk(c, 8, new, 151)
        for _ in range(3):
            b = _chunk(c, 8, new, 151)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n", [1, 150])
def test_bad_pages_and_offsets(n):
    c = Cache(160, [200, 300], 2, 128, 16, True)
    q = synth._normal((2 * n, 4, 128), 161).cuda()
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    call = lambda cu, table: fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, table, c.seqlens, n, 300, True,
                                             out=torch.full_like(q, 7.0), **c.kw)
    good, _ = call(cu, c.table)
    _check()
    for bad_page in (-1, c.pages["k"].shape[0], 2 ** 31 - 1):
        table = c.table.clone()
        table[1, 2] = bad_page
        o, _ = call(cu, table)
        _check(INVALID)
        assert torch.equal(o[:n], good[:n])
    for bad in ([0, n, 2 * n + 1], [0, n, n - 1], [-1, n, 2 * n]):
        o, _ = call(torch.tensor(bad, dtype=torch.int32, device="cuda"), c.table)
        _check(INVALID)
        skipped = o[n:] if bad[0] == 0 else o[:n]
        kept, ref = (o[:n], good[:n]) if bad[0] == 0 else (o[n:], good[n:])
        assert (skipped == 7).all() and torch.equal(kept, ref)


# ------------------------------------------------------------------------------- writing and reading


def _empty(seed, lens, H, d, page, q8):
    c = Cache(seed, lens, H, d, page, q8)
    for x in "kv":
        c.pages[x].view(torch.uint8).fill_(0x11)
        if q8:
            c.scales[x].fill_(0x22)
    return c


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,page", [(1, 16), (3, 5), (8, 1), (16, 24), (32, 256)])
def test_write_and_read(d, q8, H, page):
    new, past = [1, 0, 40, 7, 200], [0, 12, 3, 64, 1]
    lens = [a + b for a, b in zip(new, past)]
    c = _empty(200 + H, lens, H, d, page, q8)
    total, pad = sum(new), 3
    wide = synth._normal((total + pad, 2 * H + 1, d), 201, mult=3.0)  # rows further apart than they are long
    k, v = wide[:, :H], wide[:, H:2 * H]
    cu = synth.cu_seqlens_of(new)
    dev = wide.cuda()
    before = {x: (c.pages[x].clone(), c.scales[x].clone() if q8 else None) for x in "kv"}
    fa.fa_cache_write(dev[:, :H], dev[:, H:2 * H], c.pages["k"], c.pages["v"], cu.cuda(), c.table, c.seqlens, **c.kw)
    _check()
    for name, rows in (("k", k), ("v", v)):
        want = before[name][0].view(torch.uint8).cpu().numpy().copy().reshape(before[name][0].shape[:3] + (-1,))
        want_s = before[name][1].cpu().numpy().copy() if q8 else None
        if q8:
            data, s = paged.quantise(f64(rows))
        else:
            data = rows.contiguous().view(torch.uint8).numpy()
        for b in range(len(new)):
            for i in range(new[b]):
                pos = past[b] + i
                slot = (int(c.table[b, pos // page]), pos % page)
                want[slot] = data[int(cu[b]) + i]
                if q8:
                    want_s[slot] = s[int(cu[b]) + i]
        assert np.array_equal(c.pages[name].view(torch.uint8).cpu().numpy().reshape(want.shape), want)
        if q8:
            assert np.array_equal(c.scales[name].cpu().numpy(), want_s)
    # back again: the new rows as stored, rows behind the last sequence left alone
    cuk = synth.cu_seqlens_of(lens)
    outs = [torch.full((sum(lens) + pad, H, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    fa.fa_cache_read(c.pages["k"], c.pages["v"], cuk.cuda(), c.table, sum(lens) + pad, out_k=outs[0], out_v=outs[1],
                     **c.kw)
    _check()
    for rows, out in zip((k, v), outs):
        stored = paged.dequantise(*paged.quantise(f64(rows))) if q8 else f64(rows)
        assert (out[sum(lens):] == 7).all()
        for b in range(len(new)):
            at = int(cuk[b]) + past[b]
            assert np.array_equal(f64(out[at:at + new[b]]), stored[int(cu[b]):int(cu[b]) + new[b]])


@pytest.mark.parametrize("d", [64, 128])
def test_write_special_values(d):
    """Zeros, both infinities, NaN, the scale's ends, ties, and every magnitude of bf16."""
    rng = np.random.default_rng(210)
    x = rng.standard_normal((96, 2, d)) * np.exp2(rng.integers(-130, 127, (96, 2, 1)))
    x[0] = 0
    x[1, 0, 3], x[1, 1, :] = np.inf, -np.inf
    x[2, 0, 5], x[2, 1, :] = np.nan, np.nan
    x[3, 0, :], x[3, 1, 0] = 448 * 2.0 ** 60, 3e38
    x[4, 0, :4] = [448, 17, 19, 2.0 ** -10]  # ties between two codes
    x[4, 0, 4:] = 0
    x[5, 0, 0], x[5, 0, 1:] = 450, 0
    x = torch.from_numpy(x).to(torch.bfloat16)
    c = _empty(211, [96], 2, d, 16, True)
    cu = torch.tensor([0, 96], dtype=torch.int32, device="cuda")
    fa.fa_cache_write(x.cuda(), x.cuda(), c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, **c.kw)
    _check()
    codes, scales = paged.quantise(f64(x))
    row = c.table[0].cpu().numpy()
    for name in "kv":
        got = paged.gather(c.pages[name].view(torch.uint8).cpu().numpy(), row, 96)
        nan = (codes & 0x7F) == 0x7F
        assert np.array_equal((got & 0x7F) == 0x7F, nan)
        assert np.array_equal(got[~nan], codes[~nan])
        assert np.array_equal(paged.gather(c.scales[name].cpu().numpy(), row, 96), scales)
    k, _ = fa.fa_cache_read(c.pages["k"], c.pages["v"], cu, c.table, 96, **c.kw)
    assert np.array_equal(f64(k), paged.dequantise(codes, scales), equal_nan=True)


def test_write_bad_arguments_are_skipped():
    c = _empty(220, [20, 30], 2, 64, 16, False)
    x = synth._normal((12, 2, 64), 221).cuda()
    call = lambda cu, table, lens: fa.fa_cache_write(x, x, c.pages["k"], c.pages["v"], torch.tensor(
        cu, dtype=torch.int32, device="cuda"), table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    before = c.pages["k"].clone()
    bad_table = c.table.clone()
    bad_table[0] = c.pages["k"].shape[0]
    bad_table[1] = -5
    for cu, table, lens in (([0, 6, 12], bad_table, [20, 30]), ([0, 6, 12], c.table, [5, 5]),
                            ([0, 6, 12], c.table, [2 ** 31 - 1, -1]), ([0, 13, 12], c.table, [20, 30])):
        call(cu, table, lens)
        _check(INVALID)
        assert torch.equal(c.pages["k"].view(torch.uint8), before.view(torch.uint8))


def test_offsets_past_32_bits():
    """Slots beyond 4 GB into the pages of a large 8 bit cache."""
    pages, page, H, d = 9000, 256, 16, 128  # 4.7 GB of codes each
    k = torch.empty((pages, page, H, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.empty_like(k)
    ks = torch.empty((pages, page, H), dtype=torch.uint8, device="cuda")
    vs = torch.empty_like(ks)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    n = 600
    rows = synth._normal((n, 2 * H, d), 230)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    kn, vn = rows[:, :H], rows[:, H:]
    fa.fa_cache_write(kn.contiguous().cuda(), vn.contiguous().cuda(), k, v, cu, table, lens, k_scales=ks, v_scales=vs)
    kd, vd = (paged.dequantise(*paged.quantise(f64(x))) for x in (kn, vn))
    k2, v2 = fa.fa_cache_read(k, v, cu, table, n, k_scales=ks, v_scales=vs)
    assert np.array_equal(f64(k2), kd) and np.array_equal(f64(v2), vd)
    vscale = np.exp2(paged.quantise(f64(vn))[1] - 127.0)
    for m in (1, 40):
        q = synth._normal((m, H, d), 231)
        o, lse = fa.fa_fwd_paged(q.cuda(), k, v, torch.tensor([0, m], dtype=torch.int32, device="cuda"), table, lens, m,
                                 n, True, k_scales=ks, v_scales=vs)
        _close(o, lse.T, paged.attend(f64(q), kd, vd, True, 1 / math.sqrt(d), vscale), f"{m} tokens")
    _check()


# ------------------------------------------------------------------------------- as a serving loop uses them


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_serving_loop(d, q8):
    """Prompts in two pieces, then single tokens: every step written, then attended to."""
    B, hq, hkv, page, steps = 3, 4, 2, 16, [[70, 3, 129], [30, 50, 1], [1, 1, 1], [1, 1, 1], [4, 0, 2]]
    lens = [sum(s[b] for s in steps) for b in range(B)]
    c = _empty(240, lens, hkv, d, page, q8)
    have, kept = [0] * B, {x: [np.zeros((0, hkv, d))] * B for x in "kv"}
    vscale = [np.zeros((0, hkv))] * B
    for i, new in enumerate(steps):
        total = sum(new)
        q, k, v = (synth._normal((total, h, d), 250 + 10 * i + j) for j, h in enumerate((hq, hkv, hkv)))
        have = [a + b for a, b in zip(have, new)]
        cu, seqlens = synth.cu_seqlens_of(new), torch.tensor(have, dtype=torch.int32).cuda()
        fa.fa_cache_write(k.cuda(), v.cuda(), c.pages["k"], c.pages["v"], cu.cuda(), c.table, seqlens, **c.kw)
        if q8 and max(new) == min(new) == 1:
            o, lse = fa.fa_decode_paged_q8(q.cuda(), c.pages["k"], c.pages["v"], c.scales["k"], c.scales["v"], c.table,
                                           seqlens, max(have))
        else:
            o, lse = fa.fa_fwd_paged(q.cuda(), c.pages["k"], c.pages["v"], cu.cuda(), c.table, seqlens, max(new),
                                     max(have), True, **c.kw)
            lse = lse.T
        _check()
        for b in range(B):
            sl = slice(int(cu[b]), int(cu[b + 1]))
            for name, x in (("k", k), ("v", v)):
                codes, s = paged.quantise(f64(x[sl]))
                kept[name][b] = np.concatenate([kept[name][b], paged.dequantise(codes, s) if q8 else f64(x[sl])])
                if name == "v":
                    vscale[b] = np.concatenate([vscale[b], np.exp2(s - 127.0)])
            _close(o[sl], lse[sl], paged.attend(f64(q[sl]), kept["k"][b], kept["v"][b], True, 1 / math.sqrt(d),
                                                vscale[b] if q8 else None), f"step {i}, sequence {b}")


@pytest.mark.parametrize("n", [1, 130])
def test_streams_and_graphs(n):
    """On another stream than the current one's default, and two captured graphs that run
    at the same time as each other and as an eager call."""
    c = Cache(260, [3000, 500], 2, 128, 16, True)
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    qs = [synth._normal((2 * n, 8, 128), 261 + i).cuda() for i in range(3)]
    call = lambda q: fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, n, 3000, True, **c.kw)
    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    graphs, got = [], []
    for q in qs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(call(q))
        graphs.append(g)
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = call(qs[2])
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in zip(got + [eager], want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)
    del graphs


@pytest.mark.parametrize("n", [1, 150])
def test_graph_behind_other_work(n):
    """Captured behind a memset, another stream's work joined right before the call, and a write of
    the cache: the kernels' early start waits for all of it."""
    c, L = Cache(270, [700], 2, 128, 16, True), 700
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    a, b = (synth._normal((n, 8, 128), 271 + i).cuda() for i in range(2))
    new = synth._normal((n, 2, 128), 273).cuda()
    q, x = torch.empty_like(a), torch.empty_like(a)
    args = (c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, n, L, True)
    write = lambda: fa.fa_cache_write(x[:, :2], x[:, 2:4], c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, **c.kw)

    def step(side):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        x.zero_()
        with torch.cuda.stream(side):
            q.copy_(a)
            for _ in range(20):
                q.add_(b)
        x[:, :4].add_(new.repeat(1, 2, 1))
        write()
        main.wait_stream(side)
        out = fa.fa_fwd_paged(q, *args, **c.kw)
        q.zero_()  # behind the call, which has read it
        return out

    side = torch.cuda.Stream()
    want = step(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(side)
    for _ in range(5):
        got[0].fill_(9)
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    _check()
    del g


def test_launch_names():
    """The calls run the library's own kernels."""
    import ctypes
    lib = fa.load()
    c = Cache(270, [300], 2, 128, 16, True)
    lib.fa_profile_start()
    _chunk(c, 4, [3], 271)
    lib.fa_profile_stop()
    seen = {}
    for i in range(lib.fa_profile_count()):
        name, n, ms = ctypes.c_char_p(), ctypes.c_int(), ctypes.c_double()
        assert lib.fa_profile_get(i, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms)) == 0
        seen[name.value.decode()] = n.value
    assert seen["fa_paged_kernel"] == 1
