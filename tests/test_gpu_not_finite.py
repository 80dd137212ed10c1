"""A NaN among the keys comes out as NaN, wherever in a tile its key lies (the softmax takes
some keys' exponentials on other units than the rest)."""
import math

import pytest
import torch

import exact_io_aware_54_b200 as fa
from exact_io_aware_54_b200 import synth
from tests.test_gpu_paged import Cache, _check

pytestmark = pytest.mark.gpu

PLACES = [0, 2, 12, 13, 14, 15, 27, 28, 29, 30, 31, 63, 94, 126, 127, 128 + 30, 128 + 31, 298, 299]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [2, 150])
def test_nan_key_of_a_cache(n, d, q8):
    L, head = 300, 1
    c = Cache(150, [L], 2, d, 16, q8)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q = synth._normal((n, 4, d), 151).cuda()
    mine = torch.arange(4, device="cuda") // 2 == head
    pages = c.pages["k"].view(torch.uint8) if q8 else c.pages["k"]
    for at in PLACES:
        place = int(c.table[0, at // 16]), at % 16, head, 7
        old = pages[place].clone()
        pages[place] = 0xFF if q8 else math.nan
        o, lse = fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, n, L, False, **c.kw)
        _check()
        pages[place] = old
        assert o[:, mine].isnan().all() and lse[mine].isnan().all(), f"key {at}"


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [9, 15, 200])
def test_tokens_that_see_nothing_beside_nan(n, d, q8):
    """More tokens than keys, all values NaN: the first tokens see none of them."""
    L = 4
    c = Cache(155, [L, L], 2, d, 16, q8)
    c.pages["v"].view(torch.uint8).fill_(0xFF)
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    q = synth._normal((2 * n, 4, d), 156).cuda()
    o, lse = fa.fa_fwd_paged(q, c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, n, L, True, **c.kw)
    _check()
    for b in range(2):
        none = slice(b * n, b * n + n - L)
        assert (o[none] == 0).all() and (lse[:, none] == -math.inf).all()
        assert o[b * n + n - L:b * n + n].isnan().all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [2, 150])
def test_infinite_score_over_a_cache(n, d):
    """A score of +inf has no softmax: NaN, not a row that sees nothing."""
    L = 300
    c = Cache(160, [L], 1, d, 16, False)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q = synth._normal((n, 2, d), 161)
    q[..., 7] = q[..., 7].abs() + 0.125
    for at in PLACES:
        place = int(c.table[0, at // 16]), at % 16, 0, 7
        old = c.pages["k"][place].clone()
        c.pages["k"][place] = math.inf
        o, lse = fa.fa_fwd_paged(q.cuda(), c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, n, L, False)
        _check()
        c.pages["k"][place] = old
        assert o.isnan().all(), f"key {at}"


@pytest.mark.parametrize("d", [64, 128])
def test_nan_key_of_the_dense_forward(d):
    q, k, v = (x.cuda() for x in synth.prefill_inputs(170, 1, 300, 300, 2, d))
    for at in PLACES:
        bad = k.clone()
        bad[0, at, 1, 7] = math.nan
        o, _ = fa.fa_fwd(q, bad, v)
        assert fa.fa_check(fa.workspace(256, q.device, "fwd")) == 0
        assert o[:, :, 1].isnan().all(), f"key {at}"
        assert not o[:, :, 0].isnan().any()
