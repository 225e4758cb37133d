"""MXFP4 (E2M1 values, one E8M0 scale per 32) and the norms round a block, in float64.

A code's magnitudes are 0, 1/2, 1, 3/2, 2, 3, 4, 6, bit 3 its sign; a value is that times
``2^(byte - 127)``, byte 255 is NaN.  Quantisation per block of 32: scale ``2^(floor(log2
max|x|) - 2)``, at least ``2^-127``; codes nearest, ties to the even code, at most 6.
"""
from __future__ import annotations

import numpy as np

_MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_quantize64(x, scale_of=None):
    """(codes uint8 [rows][K], scale bytes uint8 [rows][K/32]) of x [rows][K]; the scales are those
    of ``scale_of`` where given."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    s = b if scale_of is None else np.asarray(scale_of, np.float64).reshape(b.shape)
    amax = np.abs(s).max(2)
    bad = ~np.isfinite(amax)
    _, e = np.frexp(np.where(bad, 0.0, amax))  # amax = m 2^e, m in [1/2, 1)
    byte = np.where(amax > 0, np.maximum(e - 3 + 127, 0), 0)
    v = np.abs(np.where(bad[:, :, None], 0.0, b)) * np.ldexp(1.0, 127 - byte)[:, :, None]
    d = np.abs(v[..., None] - _MAG)
    near = d == d.min(-1, keepdims=True)
    # one nearest, or two neighbours at the same distance: the even one of them
    lo = near.argmax(-1)
    hi = 7 - near[..., ::-1].argmax(-1)
    q = np.where(lo % 2 == 0, lo, hi) + 8 * np.signbit(np.where(bad[:, :, None], 0.0, b))
    return q.reshape(x.shape).astype(np.uint8), np.where(bad, 255, byte).astype(np.uint8)


def mx_pack(q):
    """Codes [rows][K] as bytes [rows][K/2], the lower k in the low half."""
    return (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)


def mx_values64(codes, scales):
    """Values [rows][K] of ROWS codes [rows][K/2] and scales [rows][K/32]."""
    q = np.empty((codes.shape[0], codes.shape[1] * 2), np.uint8)
    q[:, 0::2], q[:, 1::2] = codes & 15, codes >> 4
    v = np.where(q & 8, -1.0, 1.0) * _MAG[q & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=1)


def mx_round64(x, scale_of=None):
    """x rounded to MXFP4, as values."""
    q, s = mx_quantize64(x, scale_of)
    return mx_values64(mx_pack(q), s)


def mx_tiled(codes, scales):
    """The TILED layout as the header describes it, of ROWS codes and scales."""
    n, K = codes.shape[0], codes.shape[1] * 2
    J, S = -(-n // 64), -(-K // 128)
    c = np.zeros((J, S, 4, 64, 16), np.uint8)
    s = np.full((J, S, 64, 4), 127, np.uint8)
    for r in range(n):
        for g in range(K // 32):
            c[r // 64, g // 4, r // 16 % 4, 16 * (g % 4) + r % 16] = codes[r, 16 * g:16 * g + 16]
            s[r // 64, g // 4, 16 * (g % 4) + r % 16, r // 16 % 4] = scales[r, g]
    return c, s


def block_norm64(y, r=None, post_w=None, gate=None, alpha=1.0, eps=1e-6, pre_w=None, store=None):
    """(s, n): s = r + alpha gate post(y), passed through ``store`` (its rounding) where given; n its
    RMS norm with pre_w."""
    s = np.asarray(y, np.float64)
    if post_w is not None:
        s = s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * post_w
    if gate is not None:
        s = s * gate
    s = alpha * s
    if r is not None:
        s = s + r
    t = s if store is None else store(s)
    n = None if pre_w is None else t / np.sqrt((t * t).mean(1, keepdims=True) + eps) * pre_w
    return s, n
