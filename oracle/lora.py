"""Low-rank adapters beside a W4A16 projection in float64.

``y[m] = x[m] W + s_a (x[m] A_a^T) B_a^T`` with ``a = ids[m]``; a row whose id lies
outside ``[0, n)`` has the first term alone.  A is ``[n][R][K]``, B ``[n][N][R]``; adapter a
uses its first ``ranks[a]`` ranks (clamped to ``[0, R]``; None: all of them).
"""
from __future__ import annotations

import numpy as np

from .w4a16 import gemm64, silu64


def lora_rows(ids, n):
    """(adapter, its rows) for every adapter that occurs."""
    ids = np.asarray(ids, dtype=np.int64)
    for a in sorted(set(ids[(ids >= 0) & (ids < n)].tolist())):
        yield a, np.nonzero(ids == a)[0]


def lora_rank(ranks, a, R):
    return R if ranks is None else int(min(max(int(ranks[a]), 0), R))


def lora_term64(x, lora, ids) -> np.ndarray:
    """The adapters' term alone; lora = (A, B, s, ranks)."""
    A, B, s, ranks = lora
    n, R, _ = A.shape
    y = np.zeros((x.shape[0], B.shape[1]))
    for a, rows in lora_rows(ids, n):
        r = lora_rank(ranks, a, R)
        t = np.asarray(x, np.float64)[rows] @ np.asarray(A[a, :r], np.float64).T
        y[rows] = float(s[a]) * (t @ np.asarray(B[a, :, :r], np.float64).T)
    return y


def gemm_lora64(x, w, lora, ids) -> np.ndarray:
    """x W plus the adapters' term; w a (qw, sc) pair, lora None for no adapters."""
    y = gemm64(x, *w)
    return y if lora is None else y + lora_term64(x, lora, ids)


def swiglu_mlp_lora64(x, gate, up, down, lg, lu, ld, ids) -> np.ndarray:
    """The dense SwiGLU MLP with adapters on any of its projections."""
    h = silu64(gemm_lora64(x, gate, lg, ids)) * gemm_lora64(x, up, lu, ids)
    return gemm_lora64(h, down, ld, ids)
