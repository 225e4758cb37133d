"""Rows at the ends of float32's range, beside ordinary ones: the powers of two that bring a
row into f16 and back stay normal floats.  Sums of rows about 2^-118 are still normal, those
of rows about 2^121 to 2^125 still finite (the weights are small)."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
import workloads as W
from helpers import x_for_dtype, x_values
from lora_bounds import (adapters, codes, device_lora, device_weight, gemm_lora_bound, id_pattern, mlp_lora_bound)
from oracle_pool import TAU, check_elementwise, gemm_bound
from test_gpu_lora import _code, _gemm, _mlp
from test_gpu_moe_decode import _device, _reference, _run, _stacks

pytestmark = pytest.mark.gpu

ROWS = [1, 4, 8, 9, 16, 17, 64, 65, 130, 256, 600]


def _rows(M, K, dtype, seed, powers):
    """Row m is ordinary times 2^powers[m % n], its values at most 4 from zero before."""
    x = W.activations(M, K, seed)
    x = x.clamp(-4, 4) * torch.exp2(torch.tensor([powers[m % len(powers)] for m in range(M)]).float())[:, None]
    x = x_for_dtype(x, dtype).cuda()
    assert bool(torch.isfinite(x).all())
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [256, 8192])
@pytest.mark.parametrize("powers", [[-118, 0, -113], [-115.0], [121, 0, 120]])
@pytest.mark.parametrize("M", ROWS)
def test_gemm(M, powers, K, dtype):
    w = codes(K, 192, 1)
    x = _rows(M, K, dtype, 2, powers)
    y = torch.empty((M, 192), device="cuda")
    L.gemm(x, device_weight(w), y, L.new_workspace(L.gemm_workspace_bytes(M, device_weight(w), _code(dtype))))
    torch.cuda.synchronize()
    xv = x_values(x)
    check_elementwise(y.cpu().numpy(), O.gemm64(xv, *w), gemm_bound(xv, *w, TAU[dtype]), f"gemm 2^{powers} M={M}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("powers", [[-118, 0, -113], [121, 0, 120]])
@pytest.mark.parametrize("R", [16, 128])
@pytest.mark.parametrize("M", ROWS)
def test_gemm_lora(M, R, powers, dtype):
    """Without an adapter where the rows are tiny: its t would pass below the normal floats."""
    K, N, n = 256, 192, 3
    w, lo = codes(K, N, 3), adapters(n, R, K, N, 4)
    ids = id_pattern("random", M, n, 5)
    if powers[0] < 0:
        ids[np.arange(M) % len(powers) != 1] = -1
    x = _rows(M, K, dtype, 6, powers)
    y = _gemm(x, device_weight(w), device_lora(lo), torch.from_numpy(ids).cuda(), torch.float32)
    xv = x_values(x)
    check_elementwise(y.cpu().numpy(), O.gemm_lora64(xv, w, lo, ids),
                      gemm_lora_bound(xv, w, lo, ids, dtype, torch.float32), f"gemm_lora 2^{powers} M={M} R={R}")


# x about 2^-58 makes h about 2^-117
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,I", [(128, 256), (64, 8192), (1024, 512)])
@pytest.mark.parametrize("M", ROWS)
def test_swiglu_mlp(M, H, I, dtype):
    ws3 = [codes(K, N, 7 + i) for i, (K, N) in enumerate(((H, I), (H, I), (I, H)))]
    dw = [device_weight(w) for w in ws3]
    x = _rows(M, H, dtype, 10, [-58, 0, -57])
    xv = x_values(x)
    ids = np.full(M, -1, np.int32)
    ref = O.swiglu_mlp_lora64(xv, *ws3, None, None, None, ids)
    bound = mlp_lora_bound(xv, *ws3, None, None, None, ids, dtype, torch.float32)
    y = torch.empty((M, H), device="cuda")
    L.swiglu_mlp(x, *dw, y, L.new_workspace(L.swiglu_mlp_workspace_bytes(M, _code(dtype), *dw)))
    torch.cuda.synchronize()
    check_elementwise(y.cpu().numpy(), ref, bound, f"mlp M={M} H={H} I={I} {dtype}")
    y = _mlp(x, dw, [None] * 3, torch.from_numpy(ids).cuda(), torch.float32)
    check_elementwise(y.cpu().numpy(), ref, bound, f"mlp_lora M={M} H={H} I={I} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [3, 8, 40, 200])
def test_moe(M, dtype):
    H, I, E, k = 128, 192, 4, 2
    stacks = _stacks(E, H, I, 11)
    ws3, lg = _device(stacks), W.router_logits(M, E, 12)
    x = _rows(M, H, dtype, 13, [-58, 0, -57])
    ids, w = O.moe_topk(lg.numpy(), k)
    ref, bound = _reference(x_values(x), ids, w, stacks, None, dtype, torch.float32)
    dids, dwt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).float().cuda()
    y = torch.empty((M, H), device="cuda")
    L.moe_grouped(x, dids, dwt, *ws3, y, L.new_workspace(L.moe_workspace_bytes(M, k, _code(dtype), *ws3)))
    torch.cuda.synchronize()
    tiny = np.arange(M) % 3 != 1  # (the bound's float32 arithmetic passes below the normal floats there)
    bound[tiny] += 2.0 ** -10 * np.abs(ref[tiny]).max(1, keepdims=True)
    check_elementwise(y.cpu().numpy(), ref, bound, f"moe_grouped M={M} {dtype}")
    if M <= 8:
        y = _run(x, lg.cuda(), k, ws3, torch.float32, out=False)
        check_elementwise(y.cpu().numpy(), ref, bound, f"moe_decode M={M} {dtype}")
