"""Inputs and element-wise bounds for the MXFP4 tests (no test functions).

Operands enter the matrix cores exactly (E2M1 times a power of two and bf16 are exact, a
float32 value is the sum of three bf16 pieces), so a product's errors are those of its sums.
One instruction sums 32 (bf16) or 128 (fp4) terms and its accumulator in float32 or better:
its error is taken as at most 2^-20 of the sum of their magnitudes (16 float32 half-steps).
A product of K values runs K / 32 instructions a piece, three pieces for float32, or K / 128;
joining the waves' sums adds at most 16 roundings, covered by the spare instructions below.
"""
from __future__ import annotations

import numpy as np
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O

STEP = 2.0 ** -20
U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
SILU_SLOPE = 1.1  # the largest slope of z / (1 + e^-z) is 1.0998


def instructions(K, kind):
    steps = -(-K // 128)
    return 4 + {"mx": steps, "bf16": 4 * steps, "h2": 8 * steps, "f32": 12 * steps}[kind]


def weight(rng, N, K, std=0.02):
    """An MXFP4 weight: (TILED MxMatrix on the GPU, its float64 values [N][K])."""
    q, s = O.mx_quantize64(rng.standard_normal((N, K)) * std)
    return upload(q, s), O.mx_values64(O.mx_pack(q), s)


def big_weight(rng, N, K, std=0.02):
    """As weight, of uniform codes and scales in three binades (no float64 copies of a large matrix on the way)."""
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    e = int(np.floor(np.log2(std / 3)))
    s = rng.integers(126 + e, 129 + e, (N, K // 32)).astype(np.uint8)
    rows_ = L.MxMatrix(torch.as_tensor(codes).cuda(), torch.as_tensor(s).cuda(), N, K)
    return L.mx_prepack(rows_, L.mx_empty(N, K, L.MX_TILED)), O.mx_values64(codes, s)


def upload(q, s):
    c = torch.as_tensor(O.mx_pack(q)).cuda()
    rows = L.MxMatrix(c, torch.as_tensor(s).cuda(), q.shape[0], q.shape[1])
    return L.mx_prepack(rows, L.mx_empty(q.shape[0], q.shape[1], L.MX_TILED))


def rows(rng, M, K, kind, scale=1.0):
    """Activations: (what the call takes, their float64 values)."""
    x = rng.standard_normal((M, K)) * scale
    if kind == "mx":
        q, s = O.mx_quantize64(x)
        m = L.MxMatrix(torch.as_tensor(O.mx_pack(q)).cuda(), torch.as_tensor(s).cuda(), M, K)
        return m, O.mx_values64(O.mx_pack(q), s)
    t = torch.as_tensor(x).to(TORCH[kind])
    return t.cuda(), t.double().numpy()


def code_of(kind):
    return {"mx": L.MXFP4, "bf16": L.BF16, "f32": L.F32}[kind]


def gemm_bound(x, w, kind):
    return instructions(x.shape[1], kind) * STEP * (np.abs(x) @ np.abs(w).T)


def out_bound(y, b, ytype):
    return b + HALF_STEP[ytype] * (np.abs(y) + b) + 1e-37


def mlp_reference(x, gate, up, down, kind):
    """(y, bound on |y - computed| before y's own rounding)."""
    g, u = x @ gate.T, x @ up.T
    bg, bu = gemm_bound(x, gate, kind), gemm_bound(x, up, kind)
    sg = O.silu64(g)
    h = sg * u
    dh = SILU_SLOPE * bg * (np.abs(u) + bu) + np.abs(sg) * bu + 16 * U * np.abs(h)  # exp, divide, product
    if kind == "mx":
        # the computed h may lie anywhere within dh: on either side of a code's border or of its
        # block's power of two
        hq = O.mx_round64(h)
        lo, hi = np.abs(h) - dh, np.abs(h) + dh
        far = np.zeros_like(h)
        for scale_of in (np.maximum(lo, 0), hi):
            for v in (h - dh, h + dh):
                far = np.maximum(far, np.abs(O.mx_round64(v, scale_of) - hq))
        h, dh, kd = hq, far, "mx"
    elif kind == "bf16":
        dh, kd = dh + 2.0 ** -16 * (np.abs(h) + dh), "h2"
    else:
        kd = "f32"
    return h @ down.T, dh @ np.abs(down).T + instructions(h.shape[1], kd) * STEP * ((np.abs(h) + dh) @ np.abs(down).T)


def check(y, ref, bound, what):
    d = np.abs(y.double().cpu().numpy() - ref)
    worst = float((d / bound).max()) if d.size else 0.0
    assert (d <= bound).all(), f"{what}: largest error is {worst:.3g} of its bound"
    return worst
