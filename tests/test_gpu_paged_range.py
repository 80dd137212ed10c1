"""The paged attention calls over the range of the softmax: one key that outweighs all
others, beside many weak ones that together still count."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_54_b200 as fa
from exact_io_aware_54_b200 import synth
from oracle import paged
from tests._harness import f64
from tests.test_gpu_paged import Cache, _check, _close

pytestmark = pytest.mark.gpu


def _fill(c, k, v):
    """Rows k, v [n, H, d] as the keys and values of a cache's only sequence."""
    t = np.arange(c.lens[0])
    slots = c.table[0].cpu().numpy()[t // c.page], t % c.page
    for name, x in (("k", k), ("v", v)):
        x = f64(torch.from_numpy(x).to(torch.bfloat16))
        pages = c.pages[name].cpu()
        if c.q8:
            codes, s = paged.quantise(x)
            c.values[name][slots] = paged.dequantise(codes, s)
            pages = pages.view(torch.uint8)
            pages[slots] = torch.from_numpy(codes)
            pages = pages.view(torch.float8_e4m3fn)
            scales = c.scales[name].cpu()
            scales[slots] = torch.from_numpy(s)
            c.scales[name] = scales.cuda()
        else:
            c.values[name][slots] = x
            pages[slots] = torch.from_numpy(x).to(torch.bfloat16)
        c.pages[name] = pages.cuda()
    return c


def _sink_cache(seed, n, H, d, gap, q8=True, at=5):
    """One sequence of n keys: against a query of ones, key `at` scores `gap` (within 0.02) and the
    others within a few tenths of 0; values have a mean of 0.5, key `at`'s are zeros but for one."""
    c = Cache(seed, [n], H, d, 64, q8)
    rng = np.random.default_rng(seed)
    k = 0.25 * rng.standard_normal((n, H, d)) / math.sqrt(d)
    v = 0.5 + 0.25 * rng.standard_normal((n, H, d))
    eighths = round(8 * gap * math.sqrt(d))  # shared out over the dims: 8 bit codes hold them exactly
    k[at] = (eighths // d + (np.arange(d) < eighths % d)) / 8
    v[at] = 0
    v[at, :, 1] = 1
    return _fill(c, k, v)


COPIES = 150  # sequences that share the pages: whole units in a CTA, not a few tiles each


def _attend(c, hq, new, seed):
    q = (1 + 0.1 * synth._normal((new, hq, c.d), seed).double()).to(torch.bfloat16)
    many = q.repeat(COPIES, 1, 1).cuda()
    cu = torch.arange(0, COPIES * new + 1, new, dtype=torch.int32, device="cuda")
    table, lens = c.table.repeat(COPIES, 1), c.seqlens.repeat(COPIES)
    o, lse = fa.fa_fwd_paged(many, c.pages["k"], c.pages["v"], cu, table, lens, new, c.lens[0], True, **c.kw)
    _check()
    ref = c.reference(0, f64(q), True)
    for b in range(COPIES):
        sl = slice(b * new, (b + 1) * new)
        _close(o[sl], lse[:, sl].T, ref, f"{new} tokens over {c.lens[0]}, copy {b}")
    if c.q8 and new == 1:
        o2, lse2 = fa.fa_decode_paged_q8(many, c.pages["k"], c.pages["v"], c.scales["k"], c.scales["v"], table, lens,
                                         c.lens[0])
        _check()
        assert torch.equal(o, o2) and torch.equal(lse, lse2.T)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,gap", [(300, 8.0), (8192, 11.3), (16384, 12.0), (16384, 16.0), (65536, 13.0)])
def test_weak_keys_beside_a_strong_one(n, gap, d, q8):
    """Single tokens and drafted ones: the weak keys' weights are kept to their own precision."""
    c = _sink_cache(300, n, 2, d, gap, q8)
    _attend(c, 4, 1, 301)
    _attend(c, 16, 1, 302)
    _attend(c, 4, 8, 303)


def test_weak_keys_of_many_rows():
    """The same over an 8 bit cache by the kernel of many rows."""
    _attend(_sink_cache(310, 16384, 2, 128, 12.0), 4, 20, 311)
    _attend(_sink_cache(310, 16384, 2, 128, 12.0), 4, 16, 312)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("hq,new", [(2, 1), (4, 6), (4, 40)])
def test_loud_channel_of_the_queries(hq, new, q8, d):
    """Queries with one channel 2^14 times as loud as the others, which the keys leave empty:
    the scores are the quiet channels', all of the same sign."""
    n = 700
    rng = np.random.default_rng(320)
    k = rng.uniform(0, 12 / math.sqrt(d), (n, 2, 1)) * np.ones(d)
    k[..., 3] = 0
    c = _fill(Cache(321, [n], 2, d, 16, q8), k, rng.standard_normal((n, 2, d)))
    q = torch.full((new, hq, d), 1.0625, dtype=torch.bfloat16)
    q[..., 3] = 2.0 ** 14
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_paged(q.cuda(), c.pages["k"], c.pages["v"], cu, c.table, c.seqlens, new, n, True, **c.kw)
    _check()
    _close(o, lse.T, c.reference(0, f64(q), True), f"{new} tokens")
