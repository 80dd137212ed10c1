"""What the tolerances of the paged attention reference let pass (CPU): a weight split into
8 bit pieces is replayed on the host, with the stated pieces and with too few."""
import numpy as np
import pytest
import torch

from oracle import paged


def three_pieces(p):
    """p as the 8 bit kernel holds it: three e5m2 pieces, 8 and 64 times up for the later two."""
    h = torch.from_numpy(p).to(torch.float16)
    # the upper byte of the fp16 number, to the nearest (ties away from zero)
    e5 = lambda x: ((x.view(torch.int16).int() + 0x80) & 0xFF00).to(torch.int16).view(torch.float16)
    a = e5(h)
    r = (h - a) * 8
    b = e5(r)
    c = e5((r - b) * 8)
    return a.double().numpy() + b.double().numpy() / 8 + c.double().numpy() / 64


def two_pieces(p):
    """Two e4m3 pieces with one scale, largest weight 2^7: what is under 2^-17 of it is lost."""
    e4 = lambda x: x.to(torch.float8_e4m3fn).float()
    h = torch.from_numpy(p * 2.0 ** -7).float()
    a = e4(h)
    return (a + e4(h - a)).double().numpy() * 2.0 ** 7


def attend_with(split, q, k, v, scale, vs):
    """One token and head: the product takes split weights, the sum that divides the unrounded ones."""
    x = k @ q * scale
    w = np.exp(x - x.max()) * vs
    w = w / w.max() * 2.0 ** 14
    return split(w) @ (v / vs[:, None]) / (w / vs).sum()


def _case(n, gap, seed):
    rng = np.random.default_rng(seed)
    d = 16
    q = np.ones(d)
    k = 0.1 * rng.standard_normal((n, d)) / 4
    v = 0.5 + 0.25 * rng.standard_normal((n, d))
    k[3], v[3] = gap / 16, 0
    v[3, 1] = 1
    codes, s = paged.quantise(v)
    return q, k, paged.dequantise(codes, s), np.exp2(s - 127.0)


@pytest.mark.parametrize("n,gap", [(100, 3.0), (8192, 11.3), (16384, 12.0), (16384, 16.0), (65536, 13.0)])
def test_three_pieces_are_within_the_tolerance(n, gap):
    q, k, v, vs = _case(n, gap, 1)
    o, _, tol, _ = paged.attend(q[None, None], k[:, None], v[:, None], True, 1.0, vs[:, None])
    got = attend_with(three_pieces, q, k, v, 1.0, vs)
    assert (np.abs(got - o[0, 0]) <= tol[0, 0]).all()


@pytest.mark.parametrize("n,gap", [(8192, 12.0), (16384, 11.3), (16384, 12.0), (65536, 13.0)])
def test_lost_weights_are_not(n, gap):
    q, k, v, vs = _case(n, gap, 2)
    o, _, tol, _ = paged.attend(q[None, None], k[:, None], v[:, None], True, 1.0, vs[:, None])
    got = attend_with(two_pieces, q, k, v, 1.0, vs)
    assert (np.abs(got - o[0, 0]) > 2 * tol[0, 0])[2:].all()


def test_precision_of_the_pieces():
    """2^-9 + 2^-11 of a weight, and 2^-22 where the largest is 2^14: e5m2 keeps three bits a piece, the
    fp16 number they are cut from eleven; under 2^-14 the last piece's half step is 2^-17 / 64, the
    fp16 number's 2^-25."""
    p = np.exp2(np.random.default_rng(3).uniform(-40, 15, 2_000_000)).astype(np.float32).astype(np.float64)
    err = np.abs(three_pieces(p) - p)
    assert (err <= np.maximum((2.0 ** -9 + 2.0 ** -11) * p, 2.0 ** -23 + 2.0 ** -25)).all()
