"""How the paged calls behave beside one another: host threads, routes through the
kernels, workspaces, and calls with nothing to do."""
import math
import threading

import pytest
import torch

import exact_io_aware_54_b200 as fa
from exact_io_aware_54_b200 import synth
from tests._harness import f64
from tests.test_gpu_paged import INVALID, Cache, _check, _close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 40])
def test_two_host_threads_on_one_stream(new):
    """Both threads' calls go to the default stream and its workspace, and units are cut between
    CTAs, so that every call hands partial states from one launch to the next."""
    c = Cache(400, [3000, 700], 2, 128, 16, True)
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    qs = [synth._normal((2 * new, 8, 128), 401 + i).cuda() for i in range(2)]
    call = lambda q: fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, new, 3000, True, **c.kw)
    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2), [0, 0]

    def work(i):
        start.wait()
        for _ in range(40):
            out = [call(qs[i]) for _ in range(10)]
            wrong[i] += sum(not (torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])) for o, lse in out)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]
    _check()


def test_first_calls_of_two_threads():
    """A stream's workspace is made once, whichever thread comes first."""
    stream, start, got = torch.cuda.Stream(), threading.Barrier(4), []

    def work():
        with torch.cuda.stream(stream):
            start.wait()
            got.append(fa.paged_workspace().data_ptr())

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(set(got)) == 1


def _launched(call):
    """Names and counts of the library's kernels that a call launches."""
    import ctypes
    lib = fa.load()
    lib.fa_profile_start()
    call()
    lib.fa_profile_stop()
    seen = {}
    for i in range(lib.fa_profile_count()):
        name, n, ms = ctypes.c_char_p(), ctypes.c_int(), ctypes.c_double()
        assert lib.fa_profile_get(i, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms)) == 0
        if n.value:
            seen[name.value.decode()[len("fa_paged_"):]] = n.value
    return seen


FEW, FEW_JOIN, MANY, MANY_JOIN = "kernel", "merge_kernel", "chunk_kernel", "chunk_merge_kernel"


@pytest.mark.parametrize("group,keys,kernels", [
    (32, 300, [FEW, FEW_JOIN]), (33, 300, [MANY, MANY_JOIN]), (40, 128, [MANY]), (65, 129, [MANY, MANY_JOIN]),
    (32, 128, [FEW])])
def test_single_tokens_take_one_kernel(group, keys, kernels):
    """Every sequence has the group's rows, so that one kernel takes them all; units of one tile
    leave nothing to join."""
    for lens in ([keys, 7, keys - 1], [keys]):
        c = Cache(410, lens, 1, 64, 16, True)
        q = synth._normal((len(lens), group, 64), 411)
        out = []
        seen = _launched(lambda: out.extend(fa.fa_decode_paged_q8(
            q.cuda(), c.pages["k"], c.pages["v"], c.scales["k"], c.scales["v"], c.table, c.seqlens, keys)))
        _check()
        assert seen == {k: 1 for k in kernels}
        for b in range(len(lens)):
            _close(out[0][b:b + 1], out[1][b:b + 1], c.reference(b, f64(q[b:b + 1]), True), f"sequence {b}")


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("most", [1, 6, 130])
def test_chunks_longer_than_their_bound(most, causal, d, q8):
    """The first tokens are attended as what they are, the first of the chunk; the others' rows stay."""
    new, lens = [most + 7, 3, most + 200, most], [most + 40, 60, most + 90, 700]  # the third: tokens that see nothing
    c = Cache(420, lens, 2, d, 16, q8)
    cu = synth.cu_seqlens_of(new)
    q = synth._normal((sum(new), 4, d), 421)
    o = torch.full((sum(new), 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, sum(new)), 7.0, device="cuda")
    fa.fa_fwd_paged(q.cuda(), c.pages["k"], c.pages["v"], cu.cuda(), c.table, c.seqlens, most, max(lens), causal, out=o,
                    lse=lse, **c.kw)
    _check()
    for b, n in enumerate(new):
        at, cut = int(cu[b]), min(n, most)
        ref = [x[:cut] for x in c.reference(b, f64(q[at:at + n]), causal)]
        _close(o[at:at + cut], lse[:, at:at + cut].T, ref, f"sequence {b}, {cut} of {n}")
        assert (o[at + cut:at + n] == 7).all() and (lse[:, at + cut:at + n] == 7).all()


@pytest.mark.parametrize("q8", [False, True])
def test_calls_without_a_row(q8):
    """Steps in which no sequence has a token, or a key, and a batch of no sequence."""
    H, d = 2, 64
    c = Cache(430, [20, 0], H, d, 16, q8)
    before = {x: c.pages[x].view(torch.uint8).clone() for x in "kv"}
    zeros = torch.zeros(3, dtype=torch.int32, device="cuda")
    rows = torch.empty((0, H, d), dtype=torch.bfloat16, device="cuda")

    def calls():
        fa.fa_cache_write(rows, rows, c.pages["k"], c.pages["v"], zeros, c.table, c.seqlens, **c.kw)
        k, v = fa.fa_cache_read(c.pages["k"], c.pages["v"], zeros, c.table, 0, **c.kw)
        assert k.shape == v.shape == (0, H, d) and k.dtype == torch.bfloat16
        q = torch.empty((0, 4, d), dtype=torch.bfloat16, device="cuda")
        for most in (0, 5):
            o, lse = fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], zeros, c.table, c.seqlens, most, 20, True, **c.kw)
            assert o.shape == q.shape and lse.shape == (4, 0)
        if q8:
            o, lse = fa.fa_decode_paged_q8(q, c.pages["k"], c.pages["v"], c.scales["k"], c.scales["v"], c.table[:0],
                                           c.seqlens[:0], 0)
            assert o.shape == q.shape and lse.shape == (0, 4)

    assert _launched(calls) == {}
    _check()
    assert all(torch.equal(c.pages[x].view(torch.uint8), before[x]) for x in "kv")
    with pytest.raises(ValueError):  # a wrong shape is one with no row too
        fa.fa_cache_write(rows[:, :1], rows, c.pages["k"], c.pages["v"], zeros, c.table, c.seqlens, **c.kw)


def test_bounds_past_32_bits_are_refused():
    """2^32 + 20 is not a bound of 20."""
    c = Cache(440, [40], 2, 64, 16, True)
    q = synth._normal((1, 2, 64), 441).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for big in (2 ** 32, 2 ** 32 + 20, 2 ** 63 + 1, -2 ** 32 + 20):
        for most in (dict(max_seqlen_q=1, max_seqlen_k=big), dict(max_seqlen_q=big, max_seqlen_k=40)):
            with pytest.raises(ValueError, match="32 bits"):
                fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, **most, **c.kw)
        with pytest.raises(ValueError, match="32 bits"):
            fa.fa_decode_paged_q8(q, c.pages["k"], c.pages["v"], c.scales["k"], c.scales["v"], c.table, c.seqlens, big)


def _captured(call):
    """A graph of the call, what it returned, and the types of the graph's nodes."""
    from cuda.bindings import runtime
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        out = call()
    raw = runtime.cudaGraph_t(init_value=g.raw_cuda_graph())
    err, _, n = runtime.cudaGraphGetNodes(raw)
    assert err == runtime.cudaError_t.cudaSuccess
    err, nodes, n = runtime.cudaGraphGetNodes(raw, n)
    assert err == runtime.cudaError_t.cudaSuccess
    types = [runtime.cudaGraphNodeGetType(node)[1] for node in nodes[:n]]
    g.instantiate()
    return g, out, [t.name for t in types]


@pytest.mark.parametrize("new,kernels", [(1, 2), (40, 4)])
def test_captured_calls_are_their_kernels(new, kernels):
    """No other node: the kernels start early behind one another."""
    c = Cache(450, [500, 300], 2, 128, 16, True)
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    q, x = (synth._normal((2 * new, h, 128), 451 + h).cuda() for h in (8, 2))

    def call():
        fa.fa_cache_write(x, x, c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, **c.kw)
        return fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, new, 500, True, **c.kw)

    want = call()  # (also the one-time set-up, which a capture must not meet first)
    g, out, types = _captured(call)
    assert types == ["cudaGraphNodeTypeKernel"] * (1 + kernels)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    del g


@pytest.mark.parametrize("new", [1, 40])
def test_status_of_captured_calls(new):
    """With a workspace made under the capture: recorded in each replay, and cleared by the next."""
    c = Cache(460, [500, 300], 2, 128, 16, True)
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    q = synth._normal((2 * new, 8, 128), 461).cuda()
    table = c.table.clone()

    def call():
        ws = fa.paged_workspace()
        return ws, fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, table, c.seqlens, new, 500, True, ws=ws, **c.kw)

    want = fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, table, c.seqlens, new, 500, True, **c.kw)
    g, (ws, out), _ = _captured(call)
    for bad in (False, True, False):
        table.copy_(c.table)
        if bad:
            table[0, 3] = -1
        g.replay()
        assert fa.fa_check(ws) == (INVALID if bad else 0)
        assert bad or torch.equal(out[0], want[0])
    table[0, 3] = -1
    g.replay()
    table.copy_(c.table)
    g.replay()  # cleared, and nothing to record
    assert fa.fa_check(ws) == 0
    _check()
    del g


FAILED_LAUNCH = """
import ctypes, sys, torch
sys.path.insert(0, ".")
from cuda.bindings import runtime as rt
import exact_io_aware_54_b200 as fa

new = int(sys.argv[1])
bf16 = dict(dtype=torch.bfloat16, device="cuda")
pages, q, x = torch.zeros((4, 16, 1, 64), **bf16), torch.zeros((new, 1, 64), **bf16), torch.zeros((new, 1, 64), **bf16)
table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
cu, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, new], [64]))
ws, o, lse = fa.paged_workspace(), torch.empty_like(q), torch.empty((1, new), device="cuda")
torch.cuda.synchronize()
lib, p = fa.load(), lambda t: t.data_ptr()

def attend(stream):
    return lib.fa_fwd_paged(p(q), 64, p(pages), p(pages), None, None, p(cu), p(table), p(lens), p(o), p(lse), 1, 1, 1,
                            new, 4, 16, 4, new, 64, 64, 1, 0.0, p(ws), ws.numel(), stream)

def write(stream):
    return lib.fa_cache_write(p(x), p(x), 64, 64, p(cu), p(table), p(lens), p(pages), p(pages), None, None, 1, 1, new, 4,
                              16, 4, 64, p(ws), ws.numel(), stream)

assert attend(0) == 0 and write(0) == 0
torch.cuda.synchronize()
err, stream = rt.cudaStreamCreateWithFlags(rt.cudaStreamNonBlocking)
assert err == 0
assert rt.cudaStreamBeginCapture(stream, rt.cudaStreamCaptureMode.cudaStreamCaptureModeThreadLocal)[0] == 0
assert rt.cudaStreamSynchronize(stream)[0] != 0  # not allowed: the capture is now invalid, and so is a launch into it
cuda_error = [k for k, v in fa.STATUS.items() if v == "FA_ERR_CUDA"][0]
assert attend(int(stream)) == cuda_error
assert rt.cudaStreamEndCapture(stream)[0] != 0
assert write(0) == 0, "an earlier call's error"
assert attend(0) == 0 and fa.fa_check(ws) == 0
print("fine")
"""


@pytest.mark.parametrize("new", [1, 40])
def test_error_of_a_launch_is_reported_once(new):
    """A launch into a capture that has become invalid fails on the host; the next call is not blamed for it."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FAILED_LAUNCH, str(new)], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert run.stdout.strip() == "fine", run.stderr[-2000:]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens,group,kernels", [
    ([8, 8], [300, 40], 4, [FEW, FEW_JOIN]),  # 32 rows a key head
    ([11, 11], [300, 40], 3, [FEW, FEW_JOIN, MANY, MANY_JOIN]),  # 33: the bound says so, whatever the lengths
    ([8, 1], [128, 128], 4, [FEW]),  # one tile of keys: nothing to join
    ([8, 1], [129, 128], 4, [FEW, FEW_JOIN]),
    ([90, 1], [128, 20], 4, [FEW, MANY]),  # a short chunk and a long one
    ([90, 1], [129, 20], 4, [FEW, FEW_JOIN, MANY, MANY_JOIN]),
    ([3], [700], 4, [FEW, FEW_JOIN]),
    ([90], [700], 4, [MANY, MANY_JOIN]),  # one sequence: one kernel
    ([90], [90], 4, [MANY])])
def test_kernels_of_a_chunk(new, lens, group, kernels, d, q8):
    c = Cache(470, lens, 2, d, 16, q8)
    cu = synth.cu_seqlens_of(new)
    q = synth._normal((sum(new), 2 * group, d), 471)
    out = []
    seen = _launched(lambda: out.extend(fa.fa_fwd_paged(q.cuda(), c.pages["k"], c.pages["v"], cu.cuda(), c.table, c.seqlens,
                                                        max(new), max(lens), True, **c.kw)))
    _check()
    assert seen == {k: 1 for k in kernels}
    for b, n in enumerate(new):
        sl = slice(int(cu[b]), int(cu[b]) + n)
        _close(out[0][sl], out[1][:, sl].T, c.reference(b, f64(q[sl]), True), f"sequence {b}")


@pytest.mark.parametrize("d", [64, 128])
def test_single_sequence_with_a_large_bound(d):
    """A bound of many rows and a chunk of one: the kernel of many rows."""
    c = Cache(480, [300], 2, d, 16, True)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    q = synth._normal((1, 4, d), 481)
    out = []
    seen = _launched(lambda: out.extend(fa.fa_fwd_paged(q.cuda(), c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, 512,
                                                        300, True, **c.kw)))
    _check()
    assert seen == {MANY: 1, MANY_JOIN: 1}
    _close(out[0], out[1].T, c.reference(0, f64(q), True), "one token")


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("hkv", [4, 2])
def test_chunk_and_packed_forward_within_their_tolerances(hkv, q8):
    """The same keys read back and given to the packed forward: apart by no more than what both may
    be off (its roundings are the reference's: bf16 weights, the rounded sum, bf16 outputs)."""
    lens, new = [1500, 40, 513], [150, 7, 200]
    c = Cache(490, lens, hkv, 128, 16, q8)
    q = synth._normal((sum(new), 4, 128), 491)
    cu, cuk = synth.cu_seqlens_of(new), synth.cu_seqlens_of(lens).cuda()
    o, _ = fa.fa_fwd_paged(q.cuda(), c.pages["k"], c.pages["v"], cu.cuda(), c.table, c.seqlens, 200, 1500, True, **c.kw)
    k, v = fa.fa_cache_read(c.pages["k"], c.pages["v"], cuk, c.table, sum(lens), **c.kw)
    k, v = (x.repeat_interleave(4 // hkv, 1).contiguous() for x in (k, v))
    o2, _ = fa.fa_fwd_varlen(q.cuda(), k, v, cu.cuda(), cuk, 200, 1500, causal=True)
    _check()
    for b, n in enumerate(new):
        sl = slice(int(cu[b]), int(cu[b]) + n)
        tol = c.reference(b, f64(q[sl]), True)[2]
        assert (abs(f64(o[sl]) - f64(o2[sl])) <= 2 * tol).all()
