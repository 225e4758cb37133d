"""The rule in mx_plan.py against the library: the workspaces of float32 products tell streamed from
tiles, those of all types tell tiles that share columns."""
import ctypes
import math
import random

import pytest

import int4_w4a16_group_g32_amd as L
import mx_plan

CODE = {"f32": L.F32, "bf16": L.BF16, "mx": L.MXFP4}


class _W(L.MxMatrix):
    """A matrix without tensors."""

    def desc(self):
        return L.MxDesc(0x100000, 0x200000, self.rows, self.K, L.MX_TILED)


def _w(rows, K):
    return _W(None, None, rows, K, L.MX_TILED)


def _log(r, lo, hi, m):
    return max(m, int(math.exp(r.uniform(math.log(lo), math.log(hi)))) // m * m)


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
def test_workspaces_are_those_of_the_rule(kind):
    r, forms = random.Random(7), set()
    for i in range(4000):
        M, K, N = _log(r, 1, 4096, 1), _log(r, 32, 20480, 32), _log(r, 16, 65536, 16)
        if i % 2:
            M = r.randrange(17, 129)
        assert L.mx_gemm_workspace_bytes(M, CODE[kind], _w(N, K)) == mx_plan.gemm_bytes(M, K, N, kind), (M, K, N)
        forms.add(str(mx_plan.product(M, N, K, kind)))
        H, I = K, max(32, N // 32 * 32)
        H = max(32, H // 32 * 32)
        got = L.mx_swiglu_mlp_workspace_bytes(M, CODE[kind], _w(I, H), _w(I, H), _w(H, I))
        assert got == mx_plan.mlp_bytes(M, H, I, kind), (M, H, I)
    assert {"stream", "32x256", "32x256 shared", "64x256", "64x256 shared", "128x256", "128x256 shared"} <= forms
