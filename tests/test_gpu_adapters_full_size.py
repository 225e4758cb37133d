"""The adapter projections and the few-token MoE layer at the configurations' sizes (hidden
7168, intermediate 18432, 384 experts of 7168 x 2048, top-8) against the float64 oracle,
element by element: every output of the GEMMs of up to 300 rows and of the MoE layers,
sampled rows of the longest GEMM, sampled columns of the MLPs."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
import workloads as W
from helpers import rel_err, tol_for, x_for_dtype, x_values
from lora_bounds import (HALF_STEP, adapters, codes, device_lora, device_weight, gemm_lora_bound, id_pattern,
                         mlp_lora_bound)
from oracle_pool import TAU, ExpertPool, check_elementwise, mlp_bound, moe_bound_from
from test_gpu_lora import _check, _gemm, _mlp, _x
from test_gpu_moe import _random_code_stacks
from test_gpu_moe_decode import _run

pytestmark = pytest.mark.gpu

H, I = 7168, 18432


@pytest.mark.parametrize("M,N,R,n,group,kind,dtype,ytype", [
    (1, 4096, 8, 4, 32, "distinct", "f32", torch.float32),
    (16, 4096, 16, 32, 32, "random", "bf16", torch.bfloat16),
    (64, 4096, 32, 64, 64, "distinct", "bf16", torch.float32),
    (128, 4096, 16, 128, 32, "distinct", "f32", torch.float32),
    (300, 4096, 64, 8, 32, "random", "bf16", torch.bfloat16),
    (2048, 4096, 64, 8, 32, "segments", "bf16", torch.float32),
    (601, 4096, 64, 16, 128, "random", "f32", torch.float32),
])
def test_gemm_lora(M, N, R, n, group, kind, dtype, ytype):
    w, lo = codes(H, N, 1, group), adapters(n, R, H, N, 2)
    ids = id_pattern(kind, M, n, 3)
    x = _x(M, H, dtype, 4)
    dw, dl, di = device_weight(w), device_lora(lo), torch.from_numpy(ids).cuda()
    y = _gemm(x, dw, dl, di, ytype)
    assert torch.equal(y, _gemm(x, dw, dl, di, ytype))
    rows = np.arange(M) if M <= 300 else np.unique(np.concatenate([np.arange(0, M, 16), [M - 2, M - 1]]))
    xv = x_values(x)[rows]
    _check(y[torch.from_numpy(rows).cuda()], O.gemm_lora64(xv, w, lo, ids[rows]),
           gemm_lora_bound(xv, w, lo, ids[rows], dtype, ytype),
           f"gemm_lora M={M} K={H} N={N} R={R} n={n} {dtype}->{ytype}", dtype)


@pytest.fixture(scope="module")
def mlp():
    shapes = ((H, I), (H, I), (I, H))
    return ([codes(K, N, 5 + i) for i, (K, N) in enumerate(shapes)],
            [adapters(16, 16, K, N, 8 + i) for i, (K, N) in enumerate(shapes)])


@pytest.mark.parametrize("M,dtype", [(4, "f32"), (16, "bf16"), (64, "bf16"), (64, "f32"), (520, "bf16")])
def test_swiglu_mlp_lora(mlp, M, dtype):
    ws3, los = mlp
    ids = id_pattern("random", M, 16, 11)
    x = _x(M, H, dtype, 12)
    dw, dl, di = [device_weight(w) for w in ws3], [device_lora(l) for l in los], torch.from_numpy(ids).cuda()
    y = _mlp(x, dw, dl, di, torch.float32)
    assert torch.equal(y, _mlp(x, dw, dl, di, torch.float32))
    assert bool(torch.isfinite(y).all())
    rows = np.arange(M) if M <= 64 else np.arange(0, M, 13)
    cols = np.sort(np.random.default_rng(M).choice(H, size=256, replace=False))
    down = tuple(np.ascontiguousarray(t[:, cols]) for t in ws3[2])
    A, B, s, ranks = los[2]
    ld = (A, np.ascontiguousarray(B[:, cols]), s, ranks)
    xv, idr = x_values(x)[rows], ids[rows]
    ref = O.swiglu_mlp_lora64(xv, *ws3[:2], down, *los[:2], ld, idr)
    bound = mlp_lora_bound(xv, *ws3[:2], down, *los[:2], ld, idr, dtype, torch.float32)
    ys = y[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()]
    _check(ys, ref, bound, f"mlp_lora M={M} {H}/{I} {dtype}", dtype)


@pytest.fixture(scope="module")
def experts():
    cfg = W.CONFIGS["moe_decode_m64"]
    stacks, expert = _random_code_stacks(cfg, cfg.experts, cfg.K, cfg.N)
    return cfg, stacks, expert


@pytest.mark.parametrize("M,dtype,shared", [(1, "bf16", False), (8, "f32", False), (16, "bf16", True)])
def test_moe_decode(experts, M, dtype, shared):
    cfg, stacks, expert = experts
    E, k = cfg.experts, cfg.top_k
    sh = [codes(K, N, 13 + i) for i, (K, N) in enumerate(((cfg.K, cfg.N), (cfg.K, cfg.N), (cfg.N, cfg.K)))]
    dsh = [device_weight(w) for w in sh] if shared else None
    x = x_for_dtype(W.activations(M, cfg.K, 16), dtype).cuda()
    lg = W.router_logits(M, E, 17)
    y, ids, w = _run(x, lg.cuda(), k, stacks, torch.float32, dsh)
    again = _run(x, lg.cuda(), k, stacks, torch.float32, dsh)
    assert all(torch.equal(a, b) for a, b in zip((y, ids, w), again))
    cid, cw = O.moe_topk(lg.numpy(), k)
    np.testing.assert_array_equal(ids.cpu().numpy(), cid)
    xv = x_values(x)
    with ExpertPool(TAU[dtype]) as pool:
        if shared:
            ref = O.moe_shared64(xv, cid, cw, expert, E, tuple(sh), map_fn=pool)
        else:
            ref = O.moe64(xv, cid, cw, expert, E, map_fn=pool)
        bound = moe_bound_from(pool.bounds, cid, cw)
    if shared:
        bound = bound + mlp_bound(xv, *sh, TAU[dtype])
    bound = bound + HALF_STEP[torch.float32] * (np.abs(ref) + bound)
    worst = check_elementwise(y.double().cpu().numpy(), ref, bound, f"moe_decode M={M} {dtype}")
    err = rel_err(y, ref)
    print(f"moe_decode M={M} {dtype} shared={shared} relF={err:.3e} worst/bound={worst:.2e}", flush=True)
    assert err <= tol_for(dtype)
