"""fp64 reference of the paged cache operators -- TEST INFRASTRUCTURE ONLY (numpy).

The 8 bit cache format and the attention of new tokens over a paged cache, each
written out from its definition, with the error that the stated roundings of a
kernel may cause, so that a test's tolerance follows from the inputs.
"""
from __future__ import annotations

import numpy as np

E_MIN, E_MAX, E_BIAS = -60, 60, 127
# e4m3: code m < 8 stands for m 2^-9, code m >= 8 for (8 + m % 8) 2^(m // 8 - 10); 127 is NaN
E4M3 = np.array([m * 2.0 ** -9 if m < 8 else (8 + m % 8) * 2.0 ** (m // 8 - 10) for m in range(127)])


def quantise(x):
    """Rows x [..., d] -> (e4m3 codes as uint8, scale bytes as uint8), as fa_cache_write documents."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x)
    a = np.where(finite, np.abs(x), 0.0).max(-1)
    e = np.full(a.shape, E_MIN)
    for c in range(E_MIN, E_MAX):
        e = np.where(a > 448.0 * 2.0 ** c, c + 1, e)
    y = np.minimum(np.where(finite, np.abs(x), 0.0) * 2.0 ** -e[..., None].astype(np.float64), 448.0)
    hi = np.minimum(np.searchsorted(E4M3, y), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - y, y - E4M3[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(finite, code | np.where(np.signbit(x), 0x80, 0), 0x7F)
    return code.astype(np.uint8), (e + E_BIAS).astype(np.uint8)


def dequantise(codes, scales):
    codes = np.asarray(codes)
    mag = np.append(E4M3, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag) * 2.0 ** (np.asarray(scales, dtype=np.float64) - E_BIAS)[..., None]


def gather(pages, table_row, n):
    """Rows of a sequence's first n keys: [n, H, ...]."""
    page = pages.shape[1]
    t = np.arange(n)
    return pages[np.asarray(table_row)[t // page], t % page]


def attend(q, k, v, causal, scale, v_scale=None):
    """One sequence: q [n, Hq, d], k, v [L, Hkv, d] (fp64, dequantised).  Returns o
    [n, Hq, d], lse [n, Hq], and how far a kernel's o and lse may be off:

    * each weight is rounded by at most 2^-8 of itself (bf16; three e5m2 pieces of an
      fp16 number: 2^-9 + 2^-11), and the sum that divides is that of the rounded weights
      (bf16) or of the unrounded ones (pieces): 2^-8 (sum p |v| + |o|) at most;
    * with v_scale [L, Hkv] (8 bit), the pieces of a weight w = p * v_scale end at an
      error of 2^-23 + 2^-25 (half of e5m2's subnormal step, the third piece being 64 times
      up, and of fp16's), where the largest is at least 2^14: 2^-36 of it;
    * 8 bit: an element of q under 2^-14 of its row's largest is off by at most 2^-22
      of that (half of e4m3's subnormal step, 2^-10, in a piece 32 times up, where the
      largest is at least 2^7), in either kind the scores' fp32 sums by (d + 2) 2^-24
      sum |q k|; a score off by t changes o by at most 2 t sum p |v|;
    * exponentials and the final logarithm in fp32, and sums of n weights or products, in
      which a term passes through no more than n / 16 + 64 additions (a thread or a product takes
      16 keys or more at a time): (min(n, n / 16 + 48) + 16) 2^-23 relative;
    * o is stored in bf16: 2^-8 |o|.
    """
    n, hq, d = q.shape
    L, hkv = k.shape[:2]
    o, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    o_tol, lse_tol = np.full((n, hq, d), 1e-30), np.full((n, hq), 1e-30)
    if L == 0 or n == 0:
        return o, lse, o_tol, lse_tol
    seen = np.ones((n, L), bool)
    if causal:
        seen = np.arange(L)[None] <= np.arange(n)[:, None] + L - n
    rows = seen.any(-1)
    for h in range(hq):
        g = h * hkv // hq
        kh, vh, qh = k[:, g], v[:, g], q[:, h]
        x = np.where(seen, qh @ kh.T * scale, -np.inf)[rows]
        if not rows.any():
            continue
        m = x.max(-1, keepdims=True)
        p = np.exp(x - m)
        l = p.sum(-1, keepdims=True)
        o[rows, h] = p @ vh / l
        lse[rows, h] = (m + np.log(l))[:, 0]
        p = p / l
        a = p @ np.abs(vh)
        t = (d + 2) * 2.0 ** -24 * scale * (np.abs(qh[rows]) @ np.abs(kh).T).max(-1, initial=0)
        if v_scale is not None:
            t = t + scale * 2.0 ** -22 * np.abs(qh[rows]).max(-1) * np.abs(kh).sum(-1).max()
            w = p * v_scale[None, :, g]
            top = w.max(-1, keepdims=True)
            floor = np.where(seen[rows], top * 2.0 ** -36, 0.0)
            extra = floor @ (np.abs(vh) / v_scale[:, g, None])
        else:
            extra = 0.0
        t = t + (min(L, L / 16 + 48) + 16) * 2.0 ** -23
        o_abs = np.abs(o[rows, h])
        o_tol[rows, h] = 2.0 ** -8 * (a + 2 * o_abs) + extra + 2 * t[:, None] * a + 1e-30
        lse_tol[rows, h] = t + 2.0 ** -22 * np.abs(lse[rows, h]) + 1e-6
    return o, lse, o_tol, lse_tol
