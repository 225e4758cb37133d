"""GPU parity of w4a16_gemm_lora and w4a16_swiglu_mlp_lora against the float64 oracle,
element by element (bounds: lora_bounds), and what must not change a row: the other
rows, the order of the batch, a captured graph, another stream."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
import workloads as W
from helpers import rel_err, tol_for, x_for_dtype, x_values
from lora_bounds import (adapters, codes, device_lora, device_weight, gemm_lora_bound, id_pattern, mlp_lora_bound)
from oracle_pool import TAU, check_elementwise, gemm_bound

pytestmark = pytest.mark.gpu

TYPES = [("f32", torch.float32), ("bf16", torch.bfloat16), ("bf16", torch.float32), ("f32", torch.bfloat16)]


def _code(dtype):
    return L.F32 if dtype == "f32" else L.BF16


def _x(M, K, dtype, seed):
    return x_for_dtype(W.activations(M, K, seed), dtype).cuda()


def _guarded(M, N, ytype):
    """y inside a larger buffer whose last rows must stay as they were."""
    buf = torch.full((M + 2, N), 7.0, dtype=ytype, device="cuda")
    return buf, buf[:M]


def _gemm(x, w, lo, ids, ytype, ws=None, stream=None):
    M = x.shape[0]
    buf, y = _guarded(M, w.N, ytype)
    if ws is None:
        ws = L.new_workspace(L.gemm_lora_workspace_bytes(M, w, L._dtype_code(x), lo))
    L.gemm_lora(x, w, lo, ids, y, ws, stream)
    torch.cuda.synchronize()
    assert bool((buf[M:] == 7.0).all()), "rows behind the last were written"
    return y


def _mlp(x, ws3, los, ids, ytype, ws=None):
    M = x.shape[0]
    buf, y = _guarded(M, ws3[2].N, ytype)
    if ws is None:
        ws = L.new_workspace(L.swiglu_mlp_lora_workspace_bytes(M, L._dtype_code(x), *ws3, *los))
    L.swiglu_mlp_lora(x, *ws3, *los, ids, y, ws)
    torch.cuda.synchronize()
    assert bool((buf[M:] == 7.0).all()), "rows behind the last were written"
    return y


def _check(y, ref, bound, what, dtype):
    worst = check_elementwise(y.double().cpu().numpy(), ref, bound, what)
    err = rel_err(y.double(), ref)
    print(f"{what} relF={err:.3e} worst/bound={worst:.2e}", flush=True)
    if y.dtype == torch.float32:
        assert err <= tol_for(dtype)


@pytest.mark.parametrize("dtype,ytype", TYPES)
@pytest.mark.parametrize("K,N,R,n", [(64, 64, 8, 1), (256, 512, 16, 5), (1024, 192, 24, 3), (2048, 320, 64, 20),
                                     (128, 64, 72, 4), (512, 128, 256, 2)])
@pytest.mark.parametrize("M", [1, 2, 8, 9, 15, 16, 17, 37, 64, 65, 130, 300])
def test_gemm_lora_shapes(M, K, N, R, n, dtype, ytype):
    w, lo = codes(K, N, K + N), adapters(n, R, K, N, R)
    ids = id_pattern("random", M, n, M)
    x = _x(M, K, dtype, 40 + M)
    y = _gemm(x, device_weight(w), device_lora(lo), torch.from_numpy(ids).cuda(), ytype)
    xv = x_values(x)
    _check(y, O.gemm_lora64(xv, w, lo, ids), gemm_lora_bound(xv, w, lo, ids, dtype, ytype),
           f"gemm_lora M={M} K={K} N={N} R={R} n={n} {dtype}->{ytype}", dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["none", "same", "distinct", "segments", "wild"])
@pytest.mark.parametrize("M", [5, 16, 70, 260])
def test_gemm_lora_id_patterns(M, kind, dtype):
    K, N, R, n = 512, 256, 16, 70
    w, lo = codes(K, N, 1), adapters(n, R, K, N, 2)
    ids = id_pattern(kind, M, n, 3)
    x = _x(M, K, dtype, 50)
    y = _gemm(x, device_weight(w), device_lora(lo), torch.from_numpy(ids).cuda(), torch.float32)
    xv = x_values(x)
    _check(y, O.gemm_lora64(xv, w, lo, ids), gemm_lora_bound(xv, w, lo, ids, dtype, torch.float32),
           f"gemm_lora ids={kind} M={M} {dtype}", dtype)


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("M", [3, 40, 260])
def test_gemm_lora_group_sizes(M, group):
    K, N = 512, 192
    w, lo = codes(K, N, 8, group), adapters(3, 8, K, N, 9)
    ids = id_pattern("random", M, 3, 10)
    x = _x(M, K, "bf16", 11)
    y = _gemm(x, device_weight(w), device_lora(lo), torch.from_numpy(ids).cuda(), torch.bfloat16)
    xv = x_values(x)
    _check(y, O.gemm_lora64(xv, w, lo, ids), gemm_lora_bound(xv, w, lo, ids, "bf16", torch.bfloat16),
           f"gemm_lora group={group} M={M}", "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [4, 16, 100])
def test_gemm_lora_ranks_ignore_unused_slots(M, dtype):
    """Ranks past ranks[id] hold NaN; ranks beyond [0, R] are clamped."""
    K, N, R, n = 256, 128, 40, 6
    w = codes(K, N, 12)
    lo = adapters(n, R, K, N, 13, ranks=[40, 0, 1, 13, 99, -3])
    A, B = lo[0].copy(), lo[1].copy()
    for a in range(n):
        r = O.lora_rank(lo[3], a, R)
        A[a, r:] = np.nan
        B[a, :, r:] = np.nan
    ids = id_pattern("distinct", M, n, 0)
    x = _x(M, K, dtype, 14)
    y = _gemm(x, device_weight(w), device_lora((A, B, lo[2], lo[3])), torch.from_numpy(ids).cuda(), torch.float32)
    xv = x_values(x)
    _check(y, O.gemm_lora64(xv, w, lo, ids), gemm_lora_bound(xv, w, lo, ids, dtype, torch.float32),
           f"gemm_lora ranks M={M} {dtype}", dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [6, 50, 130])
def test_a_bad_adapter_or_row_stays_its_own(M, dtype):
    """An adapter of infinities and NaNs, and a row of them, change no other row's bits."""
    K, N, R, n = 256, 128, 16, 4
    w, lo = device_weight(codes(K, N, 15)), adapters(n, R, K, N, 16)
    ids = id_pattern("distinct", M, n, 0)
    ids[-1] = -1
    dev_ids = torch.from_numpy(ids).cuda()
    x = _x(M, K, dtype, 17)
    want = _gemm(x, w, device_lora(lo), dev_ids, torch.float32)
    A, B = lo[0].copy(), lo[1].copy()
    A[2, ::2], A[2, 1::2] = np.inf, np.nan
    B[2, ::2], B[2, 1::2] = np.nan, -np.inf
    got = _gemm(x, w, device_lora((A, B, lo[2], None)), dev_ids, torch.float32)
    others = torch.from_numpy(ids != 2).cuda()
    assert torch.equal(got[others], want[others])
    assert bool(torch.isnan(got[~others]).all())
    x2 = x.clone()
    x2[1] = float("nan")
    got = _gemm(x2, w, device_lora(lo), dev_ids, torch.float32)
    keep = torch.arange(M, device="cuda") != 1
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 7, 16, 33, 130])
def test_no_adapters_is_the_plain_gemm(M, dtype):
    K, N = 512, 256
    w, lo = device_weight(codes(K, N, 18)), device_lora(adapters(2, 8, K, N, 19))
    x = _x(M, K, dtype, 20)
    y = _gemm(x, w, lo, torch.full((M,), -1, dtype=torch.int32, device="cuda"), torch.float32)
    other = device_lora(adapters(5, 24, K, N, 29))
    assert torch.equal(_gemm(x, w, other, torch.full((M,), 7, dtype=torch.int32, device="cuda"), torch.float32), y)
    base = torch.empty((M, N), device="cuda")
    L.gemm(x, w, base, L.new_workspace(L.gemm_workspace_bytes(M, w, _code(dtype))))
    torch.cuda.synchronize()
    if M > 64:  # the same tiles
        assert torch.equal(y, base)
    else:       # other orders of the same sums
        qw, sc = codes(K, N, 18)
        bound = 2 * gemm_bound(x_values(x), qw, sc, TAU[dtype])
        check_elementwise(y.cpu().numpy(), base.double().cpu().numpy(), bound, "no adapters")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [3, 16, 64, 257])
def test_gemm_lora_calls_repeat_captured_and_on_another_stream(M, dtype):
    """The same bits from repeated calls on one workspace, from a replayed graph
    (eager calls of other ids in between) and on a side stream."""
    K, N, R, n = 1024, 512, 16, 8
    w, lo = device_weight(codes(K, N, 21)), device_lora(adapters(n, R, K, N, 22))
    x = _x(M, K, dtype, 23)
    ids = [torch.from_numpy(id_pattern(k, M, n, 24)).cuda() for k in ("random", "same", "none")]
    nbytes = L.gemm_lora_workspace_bytes(M, w, _code(dtype), lo)
    want = [_gemm(x, w, lo, i, torch.float32) for i in ids]
    ws = L.new_workspace(nbytes)
    for i, y in zip(ids, want):
        assert torch.equal(_gemm(x, w, lo, i, torch.float32, ws), y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(_gemm(x, w, lo, ids[0], torch.float32, ws, side), want[0])
    cur, y, gws = ids[0].clone(), torch.empty_like(want[0]), L.new_workspace(nbytes)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.gemm_lora(x, w, lo, cur, y, gws)
    for i, ref in list(zip(ids, want)) * 2:
        cur.copy_(i)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
        assert torch.equal(_gemm(x, w, lo, ids[1], torch.float32, ws), want[1])


def test_rows_do_not_depend_on_their_place():
    """A row gives the same bits wherever it stands among rows of its adapter's block count."""
    K, N, R, n, M = 512, 256, 16, 5, 64
    w, lo = device_weight(codes(K, N, 25)), device_lora(adapters(n, R, K, N, 26))
    x = _x(M, K, "f32", 27)
    ids = torch.from_numpy(id_pattern("random", M, n, 28)).cuda()
    y = _gemm(x, w, lo, ids, torch.float32)
    perm = torch.randperm(M, generator=torch.Generator().manual_seed(1)).cuda()
    assert torch.equal(_gemm(x[perm].contiguous(), w, lo, ids[perm].contiguous(), torch.float32), y[perm])


@pytest.mark.parametrize("dtype,ytype", TYPES)
@pytest.mark.parametrize("H,I,have", [(64, 64, 7), (128, 256, 7), (512, 192, 5), (256, 512, 6), (256, 1024, 3),
                                      (128, 128, 0), (128, 128, 4), (128, 320, 1)])
@pytest.mark.parametrize("M", [1, 4, 8, 9, 16, 17, 64, 100, 257])
def test_mlp_lora_shapes(M, H, I, have, dtype, ytype):
    """have: which of gate, up and down have adapters; their ranks and counts differ."""
    shapes = [(H, I), (H, I), (I, H)]
    ws3 = [codes(K, N, 30 + i) for i, (K, N) in enumerate(shapes)]
    los = [adapters(3 + i, (8, 24, 72)[i], K, N, 40 + i, ranks=None if i else [8, 3, 0])
           if have >> i & 1 else None for i, (K, N) in enumerate(shapes)]
    ids = id_pattern("random", M, 6, 33)  # some are an adapter of one projection only
    x = _x(M, H, dtype, 34)
    y = _mlp(x, [device_weight(w) for w in ws3], [device_lora(l) for l in los], torch.from_numpy(ids).cuda(), ytype)
    xv = x_values(x)
    _check(y, O.swiglu_mlp_lora64(xv, *ws3, *los, ids), mlp_lora_bound(xv, *ws3, *los, ids, dtype, ytype),
           f"mlp_lora M={M} H={H} I={I} have={have} {dtype}->{ytype}", dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [2, 16, 40, 260])
def test_mlp_lora_replays_and_reuses_its_workspace(M, dtype):
    H, I, n = 256, 512, 4
    ws3 = [device_weight(codes(K, N, 60)) for K, N in ((H, I), (H, I), (I, H))]
    los = [device_lora(adapters(n, 16, K, N, 61)) for K, N in ((H, I), (H, I), (I, H))]
    x = _x(M, H, dtype, 62)
    ids = [torch.from_numpy(id_pattern(k, M, n, 63)).cuda() for k in ("random", "same", "none")]
    want = [_mlp(x, ws3, los, i, torch.float32) for i in ids]
    nbytes = L.swiglu_mlp_lora_workspace_bytes(M, _code(dtype), *ws3, *los)
    ws, gws = L.new_workspace(nbytes), L.new_workspace(nbytes)
    cur, y = ids[0].clone(), torch.empty_like(want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.swiglu_mlp_lora(x, *ws3, *los, cur, y, gws)
    for i, ref in list(zip(ids, want)) * 2:
        cur.copy_(i)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
        assert torch.equal(_mlp(x, ws3, los, i, torch.float32, ws), ref)


def test_empty_batches_write_nothing():
    K, N = 64, 128
    w, lo = device_weight(codes(K, N, 70)), device_lora(adapters(2, 8, K, N, 71))
    d, ld = device_weight(codes(N, K, 72)), device_lora(adapters(2, 8, N, K, 73))
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    ws = L.new_workspace(256)
    L.gemm_lora(torch.empty((0, K), device="cuda"), w, lo, ids, torch.empty((0, N), device="cuda"), ws)
    L.swiglu_mlp_lora(torch.empty((0, K), device="cuda"), w, w, d, lo, lo, ld, ids,
                      torch.empty((0, K), device="cuda"), ws)
    torch.cuda.synchronize()
