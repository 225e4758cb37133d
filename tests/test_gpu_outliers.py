"""Rows with one value far above the others, in the adapter projections and the few-token
MoE layer.  x enters as f16 pieces of x 2^e, one e a row: the row's largest magnitude lies in
[2^14, 2^15), and the smallest f16 is 2^-24.  Two pieces carry a float32 value to within
2^-22 of itself plus 2^-25 there, that is 2^-39 of the row's largest; one piece carries a bf16
value (8 bits) exactly from 2^-31 of the largest on, and to within 2^-39 of it below.

The outlier sits in a weight group whose scales are zero (and meets zeros in A), so the
exact result does not contain it."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
import workloads as W
from helpers import rel_err, x_for_dtype, x_values
from lora_bounds import adapters, codes, device_lora, device_weight, gemm_lora_bound, id_pattern
from test_gpu_lora import _gemm, _mlp
from test_gpu_moe_decode import _device, _run, _stacks
from oracle_pool import check_elementwise

pytestmark = pytest.mark.gpu

C = 100  # the outlier's place


def _x(M, K, p, dtype, seed):
    x = W.activations(M, K, seed)
    x[:, C] = torch.as_tensor(np.exp2(p) * (1.0 + 0.25 * (np.arange(M) % 8)), dtype=torch.float32)
    return x_for_dtype(x, dtype).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("p", [16, 20, 24])
@pytest.mark.parametrize("M", [1, 4, 8, 16, 64, 130, 600])
def test_gemm_lora(M, p, dtype):
    K, N, n = 7168, 256, 4
    qw, sc = codes(K, N, 1)
    sc[C // 32] = 0.0
    A, B, s, _ = adapters(n, 16, K, N, 2)
    A[:, :, C] = 0.0
    ids = id_pattern("random", M, n, 3)
    x = _x(M, K, p, dtype, 4 + M)
    y = _gemm(x, device_weight((qw, sc)), device_lora((A, B, s, None)), torch.from_numpy(ids).cuda(), torch.float32)
    xv, lo = x_values(x), (A, B, s, None)
    ref = O.gemm_lora64(xv, (qw, sc), lo, ids)
    row_max = np.abs(xv).max(1, keepdims=True).astype(np.float64)
    bound = (gemm_lora_bound(xv, (qw, sc), lo, ids, dtype, torch.float32)
             + 2.0 ** -39 * row_max * O.gemm_abs64(np.ones((1, K)), qw, sc))
    worst = check_elementwise(y.cpu().numpy(), ref, bound, f"gemm_lora outlier 2^{p} M={M} {dtype}")
    err = rel_err(y, ref)
    print(f"gemm_lora outlier 2^{p} M={M} {dtype} relF={err:.3e} worst/bound={worst:.2e}", flush=True)
    if p <= 20:
        assert err <= (1e-5 if dtype == "f32" else 1e-2)


# At 2^18 (times at most 2.75) a value of x is carried to within 2^-39 2^19.5 = 2^-19.5 of about 1, so gate, up and
# their product to within 2^-18.5 = 2.7e-6 of themselves; the rest of the arithmetic stays below 1e-6.
@pytest.mark.parametrize("dtype,tol", [("f32", 1e-5), ("bf16", 1e-2)])
@pytest.mark.parametrize("M", [1, 4, 8, 16, 40])
def test_mlp_and_moe_decode(M, dtype, tol):
    H, I, E, k, p = 1024, 512, 6, 2, 18
    x = _x(M, H, p, dtype, 5)
    xv = x_values(x)
    ws3 = [codes(K, N, 6 + i) for i, (K, N) in enumerate(((H, I), (H, I), (I, H)))]
    for q, s in ws3[:2]:
        s[C // 32] = 0.0
    ids = np.full(M, -1, np.int32)
    y = _mlp(x, [device_weight(w) for w in ws3], [None] * 3, torch.from_numpy(ids).cuda(), torch.float32)
    assert rel_err(y, O.swiglu_mlp_lora64(xv, *ws3, None, None, None, ids)) <= tol
    if M > (8 if dtype == "f32" else 16):
        return
    stacks = _stacks(E, H, I, 9)
    for q, s in stacks[:2]:
        s[:, C // 32] = 0.0
    lg = W.router_logits(M, E, 10)
    y = _run(x, lg.cuda(), k, _device(stacks), torch.float32, out=False)
    cid, cw = O.moe_topk(lg.numpy(), k)
    ref = O.moe64(xv, cid, cw, lambda e: tuple((q[e], s[e]) for q, s in stacks), E)
    assert rel_err(y, ref) <= tol
