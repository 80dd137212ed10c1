"""Pins of the 8 bit cache format and the paged attention reference (CPU)."""
import numpy as np
import torch

import oracle
from oracle import paged


def test_codes_are_the_nearest_e4m3_values():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 64)) * np.exp(rng.uniform(-20, 20, (200, 1)))
    codes, scales = paged.quantise(x)
    e = scales.astype(int) - 127
    a = np.abs(x).max(-1)
    assert np.all(a <= 448 * 2.0 ** e) and np.all((a > 448 * 2.0 ** (e - 1)) | (e == -60))
    # torch's conversion rounds to nearest even as well
    y = torch.from_numpy(x / 2.0 ** e[:, None]).to(torch.float32).to(torch.float8_e4m3fn)
    assert np.array_equal(y.view(torch.uint8).numpy() & 0x7F, codes & 0x7F)
    back = paged.dequantise(codes, scales)
    # half a step: 2^-4 of the value, 2^-10 of the scale below the normal numbers
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * 2.0 ** e[:, None]))


def test_special_rows():
    x = np.zeros((6, 4))
    x[1] = [448, -449, 1, 0]
    x[2] = [np.inf, 1, np.nan, -np.inf]
    x[3] = [3e38, 1, 0, -3e38]
    x[4] = 1e-30
    codes, scales = paged.quantise(x)
    assert scales[0] == 67 and not codes[0].any()
    assert scales[1] == 128 and codes[1, 0] == codes[1, 1] & 0x7F  # 224 and 224.5 -> 224
    assert list(codes[2]) == [0x7F, codes[2, 1], 0x7F, 0x7F] and scales[2] == 127 - 8
    assert scales[3] == 187 and codes[3, 0] == 0x7E and codes[3, 3] == 0xFE
    assert scales[4] == 67 and not codes[4].any()


def test_stored_values_are_bf16_numbers():
    codes = np.arange(127, dtype=np.uint8)
    for byte in (67, 100, 127, 150, 187):
        v = paged.dequantise(codes, np.array(byte))
        t = torch.from_numpy(v)
        assert torch.equal(t.to(torch.bfloat16).double(), t)


def test_attend_against_the_dense_oracle():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((5, 6, 8)), rng.standard_normal((9, 3, 8)), rng.standard_normal((9, 3, 8))
    for causal in (False, True):
        o, lse, _, _ = paged.attend(q, k, v, causal, 0.3)
        kk, vv = np.repeat(k, 2, 1), np.repeat(v, 2, 1)
        o2, lse2 = oracle.attn_fwd(q[None], kk[None], vv[None], causal, 0.3)
        assert np.abs(o - o2[0]).max() < 1e-12 and np.abs(lse.T - lse2[0]).max() < 1e-12


def test_rows_without_a_key():
    o, lse, _, _ = paged.attend(np.ones((3, 2, 4)), np.ones((1, 1, 4)), np.ones((1, 1, 4)), True, 1.0)
    assert not o[:2].any() and np.isneginf(lse[:2]).all() and np.allclose(o[2], 1)
    o, lse, _, _ = paged.attend(np.ones((3, 2, 4)), np.ones((0, 1, 4)), np.ones((0, 1, 4)), False, 1.0)
    assert not o.any() and np.isneginf(lse).all()
