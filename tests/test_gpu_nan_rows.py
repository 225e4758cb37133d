"""A row of NaNs gives a row of NaNs at every row count, in every call, and no other row
changes a bit.  An MLP's h is such a row wherever x holds one NaN, so the down projection
meets them too."""
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import workloads as W
from helpers import x_for_dtype
from lora_bounds import adapters, codes, device_lora, device_weight, id_pattern
from test_gpu_lora import _code, _gemm, _mlp, _x
from test_gpu_moe_decode import _device, _stacks

pytestmark = pytest.mark.gpu

NAN = float("nan")
ROWS = [1, 8, 9, 16, 17, 64, 65, 130, 256, 600]  # both sides of every path's limit


def _nan_rows(M):
    return sorted({0, M // 2, M - 1})[:max(1, M - 1)]  # (two rows keep one that is well)


def _compare(run, x, nan, where):
    """run(x) with NaN in `nan` rows against run(x): those rows NaN, the others the same bits."""
    want = run(x)
    x2 = x.clone()
    for m in nan:
        x2[m, where] = NAN
    got = run(x2)
    bad = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    bad[nan] = True
    assert bool(torch.isfinite(want).all())
    assert bool(torch.isnan(got[bad]).all()), f"rows {nan} of NaNs came out as {got[bad][:, :4].tolist()}"
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [256, 8192])  # a wave a row, a workgroup a row
@pytest.mark.parametrize("M", ROWS)
def test_gemm(M, K, dtype):
    w = device_weight(codes(K, 192, 1))
    ws = L.new_workspace(L.gemm_workspace_bytes(M, w, _code(dtype)))

    def run(x):
        y = torch.empty((M, w.N), device="cuda")
        L.gemm(x, w, y, ws)
        return y

    for where in (slice(None), 5):
        _compare(run, _x(M, K, dtype, 2), _nan_rows(M), where)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,I", [(128, 256), (1024, 512), (64, 8192), (4096, 4096)])
@pytest.mark.parametrize("M", ROWS)
def test_swiglu_mlp(M, H, I, dtype):
    ws3 = [device_weight(codes(K, N, 3 + i)) for i, (K, N) in enumerate(((H, I), (H, I), (I, H)))]
    ws = L.new_workspace(L.swiglu_mlp_workspace_bytes(M, _code(dtype), *ws3))

    def run(x):
        y = torch.empty((M, H), device="cuda")
        L.swiglu_mlp(x, *ws3, y, ws)
        return y

    _compare(run, _x(M, H, dtype, 6), _nan_rows(M), 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 8, 64, 300])
def test_moe_grouped(M, dtype):
    H, I, E, k = 128, 192, 6, 2
    ws3 = _device(_stacks(E, H, I, 7))
    ids, w = torch.empty((M, k), dtype=torch.int32, device="cuda"), torch.empty((M, k), device="cuda")
    L.moe_topk(W.router_logits(M, E, 8).cuda(), k, ids, w)
    ws = L.new_workspace(L.moe_workspace_bytes(M, k, _code(dtype), *ws3))

    def run(x):
        y = torch.empty((M, H), device="cuda")
        L.moe_grouped(x, ids, w, *ws3, y, ws)
        return y

    _compare(run, _x(M, H, dtype, 9), _nan_rows(M), 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 8])
def test_moe_decode(M, dtype):
    H, I, E, k = 128, 192, 6, 2
    ws3, lg = _device(_stacks(E, H, I, 7)), W.router_logits(M, E, 8).cuda()
    ws = L.new_workspace(L.moe_decode_workspace_bytes(M, k, _code(dtype), *ws3))

    def run(x):
        y = torch.empty((M, H), device="cuda")
        L.moe_decode(x, lg, k, *ws3, y, ws)
        return y

    _compare(run, _x(M, H, dtype, 9), _nan_rows(M), 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [16, 128])  # rows by themselves up to 512 rows, or up to 128
@pytest.mark.parametrize("M", ROWS)
def test_gemm_lora(M, R, dtype):
    K, n = 256, 5
    w, lo = device_weight(codes(K, 192, 10)), device_lora(adapters(n, R, K, 192, 11))
    ids = torch.from_numpy(id_pattern("random", M, n, 12)).cuda()
    nan = _nan_rows(M)
    ids[nan[0]] = -1  # (without an adapter: the base's product alone)
    for where in (slice(None), 5):
        _compare(lambda x: _gemm(x, w, lo, ids, torch.float32), _x(M, K, dtype, 13), nan, where)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [16, 128])
@pytest.mark.parametrize("have", [7, 3, 0])  # gate, up and down; not down; none
@pytest.mark.parametrize("M", ROWS)
def test_swiglu_mlp_lora(M, have, R, dtype):
    H, I, n = 128, 320, 5
    shapes = ((H, I), (H, I), (I, H))
    ws3 = [device_weight(codes(K, N, 14 + i)) for i, (K, N) in enumerate(shapes)]
    los = [device_lora(adapters(n, R, K, N, 17 + i)) if have >> i & 1 else None for i, (K, N) in enumerate(shapes)]
    ids = torch.from_numpy(id_pattern("random", M, n, 20)).cuda()
    nan = _nan_rows(M)
    ids[nan[0]] = -1
    _compare(lambda x: _mlp(x, ws3, los, ids, torch.float32), _x(M, H, dtype, 21), nan, 5)
