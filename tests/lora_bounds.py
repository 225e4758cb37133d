"""Element-wise bounds and inputs for the low-rank-adapter tests (no test functions).

The base term keeps the bound of w4a16_gemm (oracle_pool).  The adapters' term: bf16
operands, and float32 ones as three bf16 pieces (exact) or in fused multiply-adds, so a
product is exact before it is added and every error is a rounding of a running sum, at most
u = 2^-24 of the sum of the terms' magnitudes each.  A sum of K terms, however it is
grouped, has at most K roundings: |error of t| <= K u sum |x||a|.  t is scaled (one
rounding), and its product with B sums 3 R terms, so |error| <= |s| (err(t) |b| +
(3 R + 1) u sum |t||b|).  Adding it to the base rounds once more, and y to its type.
"""
from __future__ import annotations

import numpy as np
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
from helpers import weight_from_codes
from oracle_pool import SILU_SLOPE_MAX, TAU, gemm_bound

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def term_bound(x, lora, ids):
    A, B, s, ranks = lora
    n, R, K = A.shape
    out = np.zeros((x.shape[0], B.shape[1]))
    ax = np.abs(np.asarray(x, np.float64))
    for a, rows in O.lora_rows(ids, n):
        r = O.lora_rank(ranks, a, R)
        t = ax[rows] @ np.abs(A[a, :r].astype(np.float64)).T  # at least |t|
        out[rows] = abs(float(s[a])) * ((K + 3 * R + 1) * U * t @ np.abs(B[a, :, :r].astype(np.float64)).T)
    return out


def term_abs(x, lora, ids):
    A, B, s, ranks = lora
    return O.lora_term64(np.abs(np.asarray(x, np.float64)), (np.abs(A), np.abs(B), np.abs(s), ranks), ids)


def linear_bound(x, w, lora, ids, dtype):
    b = gemm_bound(x, *w, TAU[dtype])
    if lora is not None:
        b = b + term_bound(x, lora, ids)
        b = b + U * (O.gemm_abs64(x, *w) + term_abs(x, lora, ids))
    return b


def gemm_lora_bound(x, w, lora, ids, dtype, ytype):
    b = linear_bound(x, w, lora, ids, dtype)
    return b + HALF_STEP[ytype] * (np.abs(O.gemm_lora64(x, w, lora, ids)) + b)


def carried(dh, w, lora, ids):
    """A bound dh on the error of an input, through the projection."""
    b = O.gemm_abs64(dh, *w)
    return b if lora is None else b + term_abs(dh, lora, ids)


def mlp_lora_bound(x, gate, up, down, lg, lu, ld, ids, dtype, ytype):
    g, u = O.gemm_lora64(x, gate, lg, ids), O.gemm_lora64(x, up, lu, ids)
    eg, eu = linear_bound(x, gate, lg, ids, dtype), linear_bound(x, up, lu, ids, dtype)
    s = O.silu64(g)
    h = s * u
    # silu and the product in float32: a few roundings, inside tau |h| (>= 2^-19 |h|)
    dh = SILU_SLOPE_MAX * eg * (np.abs(u) + eu) + np.abs(s) * eu + TAU[dtype] * np.abs(h)
    b = carried(dh, down, ld, ids) + linear_bound(np.abs(h) + dh, down, ld, ids, dtype)
    return b + HALF_STEP[ytype] * (np.abs(O.gemm_lora64(h, down, ld, ids)) + b)


# ---------------------------------------------------------------- inputs

def codes(K, N, seed, group=32):
    """Random code words (every nibble equally likely) and scales."""
    r = np.random.default_rng(seed)
    qw = r.integers(0, 2 ** 32, size=(K // 8, N), dtype=np.uint64).astype(np.uint32).view(np.int32)
    return qw, (r.random((K // group, N)) * 0.005 + 0.004).astype(np.float32)


def adapters(n, R, K, N, seed, ranks=None):
    """(A, B, s, ranks): float32 arrays that hold bf16 values."""
    r = np.random.default_rng(seed)

    def bf16(shape, std):
        return torch.from_numpy((r.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16).float().numpy()

    return (bf16((n, R, K), K ** -0.5), bf16((n, N, R), 0.1), (r.random(n) + 0.5).astype(np.float32),
            None if ranks is None else np.asarray(ranks, np.int32))


def device_lora(lora):
    if lora is None:
        return None
    A, B, s, ranks = lora
    return L.Lora(torch.from_numpy(A).to(torch.bfloat16).cuda(), torch.from_numpy(B).to(torch.bfloat16).cuda(),
                  torch.from_numpy(s).cuda(), None if ranks is None else torch.from_numpy(ranks).cuda())


def device_weight(w):
    return weight_from_codes(*w)


def id_pattern(kind, M, n, seed):
    r = np.random.default_rng(seed)
    if kind == "none":
        return np.full(M, -1, np.int32)
    if kind == "same":
        return np.full(M, n - 1, np.int32)
    if kind == "distinct":
        return (np.arange(M) % n).astype(np.int32)
    if kind == "segments":
        return r.integers(-1, n, M)[np.cumsum(r.random(M) < 0.15)].astype(np.int32)
    ids = r.integers(-1, n, M).astype(np.int32)  # "random"
    if kind == "wild":  # ids of no adapter in all their forms
        ids[r.random(M) < 0.5] = r.choice(np.array([n, n + 7, 2 ** 31 - 1, -2 ** 31, -2], np.int64)).astype(np.int32)
    return ids
