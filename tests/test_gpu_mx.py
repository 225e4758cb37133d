"""MXFP4 on the GPU: format bit for bit, products and the SwiGLU MLP element by element
against float64, at one row to thousands, ragged sizes, edge scales and captured graphs."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
from mx_bounds import (TORCH, big_weight, check, code_of, gemm_bound, mlp_reference, out_bound, rows, upload, weight)

pytestmark = pytest.mark.gpu


def _edges(rng, M, K):
    """Values over the whole float range, borders and zeros among them."""
    x = rng.standard_normal((M, K)) * np.ldexp(1.0, rng.integers(-140, 120, (M, K // 32)).repeat(32, 1))
    x[rng.random((M, K)) < 0.1] = 0.0
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 4.0])
    x[0, :32] = np.resize(np.concatenate([border, -border]), 32)
    x[0, 31] = 4.0
    if K > 32:
        x[-1, 32:64] = 0.0
    return x


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 7168), (3, 96), (37, 1056), (130, 256)])
def test_quantize_is_exact(M, K, xt):
    x = torch.as_tensor(_edges(np.random.default_rng(M * K), M, K)).to(TORCH[xt])
    q, s = O.mx_quantize64(x.double().numpy())
    m = L.mx_empty(M, K)
    L.mx_quantize(x.cuda(), m)
    assert np.array_equal(m.scales.cpu().numpy(), s)
    assert np.array_equal(m.codes.cpu().numpy(), O.mx_pack(q))
    for out in (torch.float32, torch.bfloat16):
        v = torch.empty((M, K), dtype=out, device="cuda")
        L.mx_dequantize(m, v)
        want = torch.as_tensor(O.mx_values64(O.mx_pack(q), s)).to(torch.float32).to(out)
        assert torch.equal(v.cpu(), want)


@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_quantize_next_to_the_borders(xt):
    """Each border between two codes and the values one step of the type beside it."""
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]).to(TORCH[xt])
    it = torch.int32 if xt == "f32" else torch.int16
    steps = [(border.view(it) + d).view(TORCH[xt]) for d in (-2, -1, 0, 1, 2)]
    v = torch.cat(steps + [-s for s in steps])  # 80 values
    x = torch.full((3, 96), 4.0, dtype=TORCH[xt])
    for r, e in enumerate((0, -120, 100)):
        x[r, :31], x[r, 32:63], x[r, 64:82] = v[:31], v[31:62], v[62:]
        x[r] = (x[r].double() * 2.0 ** e).to(TORCH[xt])
    q, s = O.mx_quantize64(x.double().numpy())
    m = L.mx_empty(3, 96)
    L.mx_quantize(x.cuda(), m)
    assert np.array_equal(m.scales.cpu().numpy(), s) and np.array_equal(m.codes.cpu().numpy(), O.mx_pack(q))


@pytest.mark.parametrize("wt", ["f32", "bf16"])
@pytest.mark.parametrize("K,N", [(32, 16), (160, 80), (1056, 208)])
def test_weights_quantize_prepack_and_come_back(K, N, wt):
    w = torch.as_tensor(_edges(np.random.default_rng(K + N), N, K).T.copy()).to(TORCH[wt])
    q, s = O.mx_quantize64(w.double().numpy().T)
    m = L.mx_empty(N, K)
    L.mx_quantize_weight(w.cuda(), m)
    assert np.array_equal(m.codes.cpu().numpy(), O.mx_pack(q)) and np.array_equal(m.scales.cpu().numpy(), s)
    t = L.mx_prepack(m, L.mx_empty(N, K, L.MX_TILED))
    c, sc = O.mx_tiled(O.mx_pack(q), s)
    assert np.array_equal(t.codes.cpu().numpy(), c.ravel()) and np.array_equal(t.scales.cpu().numpy(), sc.ravel())
    v = torch.empty((N, K), device="cuda")
    L.mx_dequantize(t, v)
    assert torch.equal(v.cpu(), torch.as_tensor(O.mx_values64(O.mx_pack(q), s)).float())


def test_blocks_that_are_not_finite():
    x = torch.ones((2, 96))
    x[0, 5], x[0, 40], x[1, 70] = float("inf"), float("nan"), -float("inf")
    m = L.mx_empty(2, 96)
    L.mx_quantize(x.cuda(), m)
    assert m.scales.cpu().tolist() == [[255, 255, 125], [125, 125, 255]]
    assert m.codes[0, :32].eq(0).all() and m.codes[1, 32:].eq(0).all()
    v = torch.empty((2, 96), device="cuda")
    L.mx_dequantize(m, v)
    assert v.isnan().cpu().tolist() == [[True] * 64 + [False] * 32, [False] * 64 + [True] * 32]


GEMM_SHAPES = [(1, 256, 512), (2, 32, 16), (5, 96, 48), (8, 2304, 1040), (16, 1056, 272), (17, 160, 80), (37, 2304, 784),
               (64, 1056, 528), (100, 512, 256), (129, 416, 336), (200, 1152, 1168), (300, 640, 512)]


@pytest.mark.parametrize("kind,yt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("mx", "f32"), ("mx", "bf16")])
@pytest.mark.parametrize("M,K,N", GEMM_SHAPES)
def test_gemm(M, K, N, kind, yt):
    rng = np.random.default_rng(1000 * M + K + N)
    w, wv = weight(rng, N, K)
    x, xv = rows(rng, M, K, kind)
    y = torch.full((M, N), float("nan"), dtype=TORCH[yt], device="cuda")
    ws = L.new_workspace(L.mx_gemm_workspace_bytes(M, code_of(kind), w))
    L.mx_gemm(x, w, y, ws)
    ref = xv @ wv.T
    worst = check(y, ref, out_bound(ref, gemm_bound(xv, wv, kind), TORCH[yt]), f"{M}x{K}x{N} {kind}")
    print(f"mx_gemm {M}x{K}x{N} {kind}->{yt}: {worst:.3f} of the bound", flush=True)
    again = torch.empty_like(y)
    L.mx_gemm(x, w, again, ws)
    assert torch.equal(y, again)


# widths at which a workgroup of a few rows takes one, two, four to six blocks of columns
WIDE = [(1, 160, 4112), (4, 96, 18448), (7, 288, 8208), (8, 160, 16400), (13, 96, 20400), (16, 416, 4112)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("M,K,N", WIDE)
def test_gemm_of_few_rows_and_many_columns(M, K, N, kind):
    rng = np.random.default_rng(M + N)
    w, wv = weight(rng, N, K)
    x, xv = rows(rng, M, K, kind)
    y = torch.full((M + 1, N), 7.0, device="cuda")
    L.mx_gemm(x, w, y[:M], L.new_workspace(L.mx_gemm_workspace_bytes(M, code_of(kind), w)))
    check(y[:M], xv @ wv.T, out_bound(xv @ wv.T, gemm_bound(xv, wv, kind), torch.float32), f"{M}x{K}x{N} {kind}")
    assert y[M].eq(7.0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("M,H,I", [(3, 96, 18464), (6, 160, 4128), (16, 96, 18464), (2, 64, 10272), (11, 32, 24608)])
def test_swiglu_mlp_of_few_rows_and_a_wide_intermediate(M, H, I, kind):
    rng = np.random.default_rng(M + H + I)
    (g, gv), (u, uv), (d, dv) = weight(rng, I, H, 0.2), weight(rng, I, H, 0.2), weight(rng, H, I, 0.06)
    x, xv = rows(rng, M, H, kind)
    y = torch.empty((M, H), device="cuda")
    L.mx_swiglu_mlp(x, g, u, d, y, L.new_workspace(L.mx_swiglu_mlp_workspace_bytes(M, code_of(kind), g, u, d)))
    ref, b = mlp_reference(xv, gv, uv, dv, kind)
    check(y, ref, out_bound(ref, b, torch.float32), f"{M}x{H}x{I} {kind}")


# shapes whose tiles share their columns' K among workgroups (the workspace holds their sums), in
# tiles of 32, 64 and 128 rows, one row tile and several, K that ends inside a stage and a unit
SHARED = [(17, 7136, 4112), (32, 7136, 4112), (50, 7168, 4112), (64, 7136, 4112), (100, 6176, 4112), (150, 2336, 784)]
# several blocks of 16 rows streamed (the first of MXFP4 rows in shared tiles), and unshared tiles of few rows
OTHERS = [(50, 7168, 2576), (20, 7168, 2576), (17, 4256, 4112), (64, 4000, 4112), (100, 4096, 2064), (17, 288, 65552),
          (40, 544, 65552)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("M,K,N", SHARED + OTHERS)
def test_gemm_of_shared_tiles(M, K, N, kind):
    rng = np.random.default_rng(M + K + N)
    w, wv = big_weight(rng, N, K)
    x, xv = rows(rng, M, K, kind)
    size = L.mx_gemm_workspace_bytes(M, code_of(kind), w)
    assert size >= 2 * M * N * 4 or (M, K, N) in OTHERS  # at least two workgroups' sums
    y = torch.full((M + 1, N), 7.0, device="cuda")
    ws = L.new_workspace(size)
    L.mx_gemm(x, w, y[:M], ws)
    ref = xv @ wv.T
    check(y[:M], ref, out_bound(ref, gemm_bound(xv, wv, kind), torch.float32), f"{M}x{K}x{N} {kind}")
    assert y[M].eq(7.0).all()
    again = torch.empty((M, N), device="cuda")
    L.mx_gemm(x, w, again, ws)
    assert torch.equal(y[:M], again)


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("M,H,I", [(20, 2048, 4128), (50, 2048, 4128), (100, 1024, 4128), (30, 4128, 2080),
                                   (40, 7168, 4128), (72, 6176, 4128)])
def test_swiglu_mlp_of_shared_tiles(M, H, I, kind):
    """One product in tiles or both, h handed on in either's form."""
    rng = np.random.default_rng(M + H + I)
    (g, gv), (u, uv), (d, dv) = big_weight(rng, I, H), big_weight(rng, I, H), big_weight(rng, H, I)
    x, xv = rows(rng, M, H, kind)
    y = torch.empty((M, H), device="cuda")
    size = L.mx_swiglu_mlp_workspace_bytes(M, code_of(kind), g, u, d)
    L.mx_swiglu_mlp(x, g, u, d, y, L.new_workspace(size))
    ref, b = mlp_reference(xv, gv, uv, dv, kind)
    check(y, ref, out_bound(ref, b, torch.float32), f"{M}x{H}x{I} {kind}")


def test_tiles_of_twice_the_columns():
    """Many MXFP4 rows and columns: 128 x 512 tiles, and 128 x 256 of h; ragged on both sides."""
    rng = np.random.default_rng(5)
    M, K, N = 1030, 160, 9232
    w, wv = big_weight(rng, N, K)
    x, xv = rows(rng, M, K, "mx")
    y = torch.full((M + 1, N), 7.0, device="cuda")
    L.mx_gemm(x, w, y[:M], L.new_workspace(L.mx_gemm_workspace_bytes(M, L.MXFP4, w)))
    check(y[:M], xv @ wv.T, out_bound(xv @ wv.T, gemm_bound(xv, wv, "mx"), torch.float32), "gemm")
    assert y[M].eq(7.0).all()
    M, H, I = 1030, 96, 9248
    (g, gv), (u, uv), (d, dv) = big_weight(rng, I, H, 0.2), big_weight(rng, I, H, 0.2), big_weight(rng, H, I)
    x, xv = rows(rng, M, H, "mx")
    y = torch.empty((M, H), device="cuda")
    L.mx_swiglu_mlp(x, g, u, d, y, L.new_workspace(L.mx_swiglu_mlp_workspace_bytes(M, L.MXFP4, g, u, d)))
    ref, b = mlp_reference(xv, gv, uv, dv, "mx")
    check(y, ref, out_bound(ref, b, torch.float32), "mlp")


# more tiles than the card has compute units, and not a multiple: the last columns go in smaller tiles
@pytest.mark.parametrize("kind,M,K,N", [("f32", 2060, 1312, 4112), ("bf16", 2060, 1312, 4112), ("bf16", 260, 928, 23056),
                                        ("mx", 2060, 4128, 7824), ("mx", 1030, 4128, 16912)])
def test_gemm_of_a_ragged_last_round(kind, M, K, N):
    rng = np.random.default_rng(M + K + N)
    w, wv = big_weight(rng, N, K)
    x, xv = rows(rng, M, K, kind)
    y = torch.full((M + 1, N), 7.0, device="cuda")
    L.mx_gemm(x, w, y[:M], L.new_workspace(L.mx_gemm_workspace_bytes(M, code_of(kind), w)))
    ref = xv @ wv.T
    check(y[:M], ref, out_bound(ref, gemm_bound(xv, wv, kind), torch.float32), f"{M}x{K}x{N} {kind}")
    assert y[M].eq(7.0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
def test_swiglu_mlp_of_a_ragged_last_round(kind):
    rng = np.random.default_rng(9)
    M, H, I = 1030, 1312, 7200
    (g, gv), (u, uv), (d, dv) = big_weight(rng, I, H), big_weight(rng, I, H), big_weight(rng, H, I)
    x, xv = rows(rng, M, H, kind)
    y = torch.empty((M, H), device="cuda")
    L.mx_swiglu_mlp(x, g, u, d, y, L.new_workspace(L.mx_swiglu_mlp_workspace_bytes(M, code_of(kind), g, u, d)))
    ref, b = mlp_reference(xv, gv, uv, dv, kind)
    check(y, ref, out_bound(ref, b, torch.float32), f"{M}x{H}x{I} {kind}")


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_gemm_scales_over_the_whole_range(M, kind):
    """Blocks 2^-60 to 2^60 apart inside a dot product, and rows far from one another."""
    rng = np.random.default_rng(M)
    K, N = 384, 160
    q, s = O.mx_quantize64(rng.standard_normal((N, K)))
    s = rng.integers(127 - 30, 127 + 30, s.shape).astype(np.uint8)
    w, wv = upload(q, s), O.mx_values64(O.mx_pack(q), s)
    x, xv = rows(rng, M, K, kind, np.ldexp(1.0, rng.integers(-30, 30, (M, K // 32))).repeat(32, 1))
    y = torch.empty((M, N), device="cuda")
    L.mx_gemm(x, w, y, L.new_workspace(L.mx_gemm_workspace_bytes(M, code_of(kind), w)))
    check(y, xv @ wv.T, out_bound(xv @ wv.T, gemm_bound(xv, wv, kind), torch.float32), kind)


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("M", [5, 50, 270])
def test_rows_and_columns_that_are_not_finite_stay_alone(M, kind):
    rng = np.random.default_rng(M)
    K, N = 288, 112
    q, s = O.mx_quantize64(rng.standard_normal((N, K)))
    s[7, 3] = 255
    w = upload(q, s)
    clean = np.array(s)
    clean[7, 3] = 127
    wv = O.mx_values64(O.mx_pack(q), clean)
    x, xv = rows(rng, M, K, kind)
    if kind == "mx":
        x.scales[2, 4] = 255
    else:
        x[2, 130] = float("nan")
    y = torch.empty((M, N), device="cuda")
    L.mx_gemm(x, w, y, L.new_workspace(L.mx_gemm_workspace_bytes(M, code_of(kind), w)))
    bad = y.isnan().cpu()
    assert bad[2].all() and bad[:, 7].all()
    bad[2], bad[:, 7] = False, False
    assert not bad.any()
    keep_m, keep_n = [m for m in range(M) if m != 2], [n for n in range(N) if n != 7]
    xv = xv[keep_m]
    check(y[keep_m][:, keep_n], xv @ wv[keep_n].T,
          out_bound(xv @ wv[keep_n].T, gemm_bound(xv, wv[keep_n], kind), torch.float32), kind)


MLP_SHAPES = [(1, 256, 512), (3, 96, 160), (4, 1056, 2304), (16, 512, 1056), (33, 288, 224), (64, 1024, 2304),
              (150, 416, 352), (300, 512, 640)]


@pytest.mark.parametrize("kind,yt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("mx", "bf16")])
@pytest.mark.parametrize("M,H,I", MLP_SHAPES)
def test_swiglu_mlp(M, H, I, kind, yt):
    rng = np.random.default_rng(M + H + I)
    (g, gv), (u, uv), (d, dv) = weight(rng, I, H, 0.06), weight(rng, I, H, 0.06), weight(rng, H, I, 0.06)
    x, xv = rows(rng, M, H, kind)
    y = torch.full((M, H), float("nan"), dtype=TORCH[yt], device="cuda")
    ws = L.new_workspace(L.mx_swiglu_mlp_workspace_bytes(M, code_of(kind), g, u, d))
    L.mx_swiglu_mlp(x, g, u, d, y, ws)
    ref, b = mlp_reference(xv, gv, uv, dv, kind)
    worst = check(y, ref, out_bound(ref, b, TORCH[yt]), f"{M}x{H}x{I} {kind}")
    print(f"mx_swiglu_mlp {M}x{H}x{I} {kind}->{yt}: {worst:.3f} of the bound", flush=True)
    again = torch.empty_like(y)
    L.mx_swiglu_mlp(x, g, u, d, again, ws)
    assert torch.equal(y, again)


def test_zero_rows_do_nothing():
    rng = np.random.default_rng(0)
    w, _ = weight(rng, 64, 64)
    ws = L.new_workspace(256)
    y = torch.empty((0, 64), device="cuda")
    L.mx_gemm(torch.empty((0, 64), device="cuda"), w, y, ws)
    L.mx_gemm(L.mx_empty(0, 64), w, y, ws)
    L.mx_swiglu_mlp(torch.empty((0, 64), device="cuda"), w, w, w, y, ws)
    L.mx_quantize(y, L.mx_empty(0, 64))
    torch.cuda.synchronize()


@pytest.mark.parametrize("yt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 40])
def test_empty_sums_are_zeros(M, yt):
    """K of 0, and an MLP whose intermediate has no columns."""
    ws = L.new_workspace(256)
    w, d = L.mx_empty(48, 0, L.MX_TILED), L.mx_empty(64, 0, L.MX_TILED)
    g = L.mx_empty(0, 64, L.MX_TILED)
    for x in (torch.empty((M, 0), device="cuda"), L.mx_empty(M, 0)):
        y = torch.full((M, 48), 7.0, dtype=yt, device="cuda")
        L.mx_gemm(x, w, y, ws)
        assert not y.any()
    for x in (torch.ones((M, 64), device="cuda"), L.mx_empty(M, 64)):
        y = torch.full((M, 64), 7.0, dtype=yt, device="cuda")
        L.mx_swiglu_mlp(x, g, g, d, y, ws)
        assert not y.any()


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("M", [4, 70, 260])
def test_captured_and_replayed(M, kind):
    """A captured MLP gives the eager bits on every replay, on new inputs and between eager calls."""
    rng = np.random.default_rng(M)
    H, I = 512, 736
    (g, _), (u, _), (d, _) = weight(rng, I, H), weight(rng, I, H), weight(rng, H, I)
    x, _ = rows(rng, M, H, kind)
    y = torch.empty((M, H), device="cuda")
    ws = L.new_workspace(L.mx_swiglu_mlp_workspace_bytes(M, code_of(kind), g, u, d))
    other = L.new_workspace(ws.numel())
    L.mx_swiglu_mlp(x, g, u, d, y, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.mx_swiglu_mlp(x, g, u, d, y, ws)
    for i in range(3):
        new, _ = rows(np.random.default_rng(50 + i), M, H, kind)
        if kind == "mx":
            x.codes.copy_(new.codes), x.scales.copy_(new.scales)
        else:
            x.copy_(new)
        want = torch.empty_like(y)
        L.mx_swiglu_mlp(x, g, u, d, want, other)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_two_streams_with_their_own_workspaces():
    rng = np.random.default_rng(9)
    w, _ = weight(rng, 1040, 2304)
    xs = [rows(rng, 48, 2304, "bf16")[0] for _ in range(2)]
    n = L.mx_gemm_workspace_bytes(48, L.BF16, w)
    wss, ys, want = [L.new_workspace(n) for _ in xs], [torch.empty((48, 1040), device="cuda") for _ in xs], []
    for x in xs:
        want.append(torch.empty((48, 1040), device="cuda"))
        L.mx_gemm(x, w, want[-1], wss[0])
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, x, y, ws in zip(streams, xs, ys, wss):
            L.mx_gemm(x, w, y, ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))


def test_weights_quantized_on_another_stream():
    """Their intermediate rows are freed while that stream still works: the current stream's tensors are not put there."""
    w = torch.randn((4096, 4096), device="cuda")
    want = L.mx_quantize_to_weight(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [L.mx_quantize_to_weight(w, side) for _ in range(3)]
    other = [torch.full((4096 * 2048,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(g.codes, want.codes) and torch.equal(g.scales, want.scales) for g in got)
    assert all(o.eq(255).all() for o in other)


def test_rows_behind_the_last_stay_as_they_were():
    rng = np.random.default_rng(3)
    w, _ = weight(rng, 272, 160)
    for kind in ("f32", "bf16", "mx"):
        for M in (5, 21, 70, 140):
            x, _ = rows(rng, M, 160, kind)
            buf = torch.full((M + 3, 272), 7.0, device="cuda")
            L.mx_gemm(x, w, buf[:M], L.new_workspace(L.mx_gemm_workspace_bytes(M, code_of(kind), w)))
            assert buf[M:].eq(7.0).all()


def test_a_layer_as_it_is_served():
    """Norm to MXFP4 rows, SwiGLU MLP on them, post-norm with gate and residual: a run of the calls
    together, against float64 from the same inputs at each border."""
    rng = np.random.default_rng(21)
    M, H, I = 19, 512, 1056
    (g, gv), (u, uv), (d, dv) = weight(rng, I, H, 0.06), weight(rng, I, H, 0.06), weight(rng, H, I, 0.06)
    t = lambda *s: torch.as_tensor(rng.standard_normal(s)).to(torch.bfloat16).cuda()  # noqa: E731
    y0, r0, pre, post, gate = t(M, H), t(M, H), t(H), t(H), t(M, H)
    n, r1 = L.mx_empty(M, H), torch.empty_like(r0)
    L.block_norm(y0, r0, r1, n, pre_w=pre)
    y1 = torch.empty((M, H), dtype=torch.bfloat16, device="cuda")
    L.mx_swiglu_mlp(n, g, u, d, y1, L.new_workspace(L.mx_swiglu_mlp_workspace_bytes(M, L.MXFP4, g, u, d)))
    r2, n2 = torch.empty_like(r0), torch.empty_like(r0)
    L.block_norm(y1, r1, r2, n2, pre_w=pre, post_w=post, gate=gate, alpha=0.5)
    f = lambda v: v.double().cpu().numpy()  # noqa: E731
    xv = O.mx_values64(n.codes.cpu().numpy(), n.scales.cpu().numpy())
    _, nn = O.block_norm64(f(y0), f(r0), pre_w=f(pre), store=lambda s: f(torch.as_tensor(s).float().bfloat16()))
    assert np.array_equal(xv, O.mx_round64(nn))
    ref, b = mlp_reference(xv, gv, uv, dv, "mx")
    check(y1, ref, out_bound(ref, b, torch.bfloat16), "mlp")
    s, _ = O.block_norm64(f(y1), f(r1), f(post), f(gate), 0.5)
    check(r2, s, 2.0 ** -8 * np.abs(s) + 2.0 ** -18 * (np.abs(s) + np.abs(f(r1))), "residual")
    _, n2v = O.block_norm64(f(r2), pre_w=f(pre))
    check(n2, n2v, (2.0 ** -8 + 2.0 ** -18) * np.abs(n2v) + 1e-30, "norm")
