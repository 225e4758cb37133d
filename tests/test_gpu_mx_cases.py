"""MXFP4 on the GPU: calls that lie beside those of test_gpu_mx.py."""
import ctypes

import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import mx_plan
import oracle as O
from mx_bounds import check, code_of, gemm_bound, out_bound, rows, upload

pytestmark = pytest.mark.gpu


def _on_gpu(a):
    return torch.as_tensor(a).cuda()


@pytest.mark.parametrize("N,K", [(64, 128), (80, 160), (512, 2048)])
def test_prepack_into_the_source_descriptor(N, K):
    """`out` may be `src`: the kernel reads the tensors the descriptor named before the call."""
    rng = np.random.default_rng(N)
    q, s = rng.integers(0, 256, (N, K // 2), dtype=np.uint8), rng.integers(0, 256, (N, K // 32), dtype=np.uint8)
    codes, scales = _on_gpu(q), _on_gpu(s)
    dst = L.mx_empty(N, K, L.MX_TILED)
    dst.codes.fill_(0x55), dst.scales.fill_(0x55)
    d = L.MxDesc(codes.data_ptr(), scales.data_ptr(), N, K, L.MX_ROWS)
    st = L.load_library().w4a16_mx_prepack(ctypes.byref(d), dst.codes.data_ptr(), dst.codes.numel(),
                                           dst.scales.data_ptr(), dst.scales.numel(), ctypes.byref(d),
                                           torch.cuda.current_stream().cuda_stream)
    assert st == L.OK
    assert (d.codes, d.scales, d.rows, d.K, d.layout) == (dst.codes.data_ptr(), dst.scales.data_ptr(), N, K, L.MX_TILED)
    c, sc = O.mx_tiled(q, s)
    assert np.array_equal(dst.codes.cpu().numpy(), c.ravel()) and np.array_equal(dst.scales.cpu().numpy(), sc.ravel())


def _gemm(x, w, N, kind):
    M = x.rows if kind == "mx" else x.shape[0]
    y = torch.full((M, N), 7.0, device="cuda")
    L.mx_gemm(x, w, y, L.new_workspace(L.mx_gemm_workspace_bytes(M, code_of(kind), w)))
    return y


# M, K, N: the forms of a float32 product (streamed by 4, 8 and 16 rows and in blocks; tiles of 32, 64 and
# 128 rows, whole and shared; a last round in smaller tiles)
FORMS = [(1, 256, 512), (4, 96, 18448), (7, 288, 8208), (16, 416, 4112), (37, 2304, 784), (17, 7136, 4112), (40, 544, 65552),
         (64, 7136, 4112), (100, 6176, 4112), (300, 640, 512), (17, 544, 65552), (300, 64, 512), (2060, 1312, 4112)]
SMALL = FORMS[:-1]


def test_the_shapes_have_these_forms():
    assert {str(mx_plan.product(M, N, K, "f32")) for M, K, N in FORMS} == {
        "stream", "32x256", "32x256 shared", "64x256", "64x256 shared", "128x256", "128x256 shared", "128x256 rest 64x256"}


@pytest.mark.parametrize("M,K,N", FORMS)
def test_float32_rows_keep_every_bit(M, K, N):
    """One value a row and weights that are powers of two: y is that value, shifted.  All three pieces
    are needed for its 24 bits, and every sum on the way is exact."""
    rng = np.random.default_rng(M + K + N)
    q = rng.choice(np.array([1, 2, 4, 6], np.uint8), (N, K)) + 8 * rng.integers(0, 2, (N, K), dtype=np.uint8)
    s = rng.integers(110, 140, (N, K // 32)).astype(np.uint8)
    wv = O.mx_values64(O.mx_pack(q), s)
    x = np.zeros((M, K), np.float32)
    k = rng.integers(0, K, M)
    # odd last bits: a value of all 24
    v = np.ldexp((rng.integers(1 << 22, 1 << 23, M) * 2 + 1).astype(np.float64), rng.integers(-40, 40, M)) * rng.choice([-1, 1], M)
    x[np.arange(M), k] = v
    assert np.array_equal(x[np.arange(M), k].astype(np.float64), v)
    y = _gemm(_on_gpu(x), upload(q, s), N, "f32")
    assert torch.equal(y.cpu(), torch.as_tensor((v[:, None] * wv[:, k].T).astype(np.float32)))


@pytest.mark.parametrize("M,H,I", [(1, 96, 160), (4, 64, 18464), (8, 160, 4128), (16, 96, 2080), (37, 2304, 784 + 16),
                                   (64, 2048, 4128), (150, 416, 352), (300, 512, 640)])
def test_float32_rows_keep_every_bit_through_the_mlp(M, H, I):
    """gate = 32 (its silu is 32), up one value of 24 bits, down one weight: y is that value, shifted."""
    rng = np.random.default_rng(M + H + I)
    one = lambda N, K, at, c: _one_hot(N, K, at, c, 127)  # noqa: E731
    x = np.zeros((M, H), np.float32)
    x[:, 0] = 16.0
    v = np.ldexp((rng.integers(1 << 22, 1 << 23, M) * 2 + 1).astype(np.float64), -23)
    x[:, 1] = v
    i, j = np.zeros(I, int), np.ones(I, int)
    g, u = one(I, H, i, 4), one(I, H, j, 2)  # x[0] * 2, x[1] * 1
    at = rng.integers(0, I, H)
    d = one(H, I, at, 1)  # half of h[at]
    y = torch.empty((M, H), device="cuda")
    L.mx_swiglu_mlp(_on_gpu(x), g, u, d, y, L.new_workspace(L.mx_swiglu_mlp_workspace_bytes(M, L.F32, g, u, d)))
    assert torch.equal(y.cpu(), torch.as_tensor(np.repeat(16 * v[:, None], H, 1).astype(np.float32)))


def _one_hot(N, K, at, code, byte):
    q = np.zeros((N, K), np.uint8)
    q[np.arange(N), at] = code
    return upload(q, np.full((N, K // 32), byte, np.uint8))


@pytest.mark.parametrize("M,K,N", SMALL)
def test_float32_rows_near_the_smallest(M, K, N):
    """Values near 2^-120, whose third piece bf16's smallest step, 2^-133, rounds: each is off by at most
    2^-134.  The weights bring them back to the ordinary range."""
    rng = np.random.default_rng(M + K)
    q, s = rng.integers(0, 16, (N, K)).astype(np.uint8), rng.integers(232, 238, (N, K // 32)).astype(np.uint8)
    wv = O.mx_values64(O.mx_pack(q), s)
    x = torch.as_tensor(np.ldexp(rng.standard_normal((M, K)), -120)).float()
    y, xv = _gemm(x.cuda(), upload(q, s), N, "f32"), x.double().numpy()
    ref = xv @ wv.T
    check(y, ref, out_bound(ref, gemm_bound(xv, wv, "f32") + 2.0 ** -134 * np.abs(wv).sum(1), torch.float32), "small rows")


@pytest.mark.parametrize("xe,we", [(100, -110), (-100, 110), (-118, 118), (110, -120)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_scales_at_both_ends_of_the_range(M, kind, xe, we):
    """Very large rows on very small weights (subnormal ones among them), and the other way round."""
    rng = np.random.default_rng(M + abs(we))
    K, N = 416, 160
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    s = np.clip(rng.integers(127 + we - 8, 127 + we + 6, (N, K // 32)), 0, 251).astype(np.uint8)
    wv = O.mx_values64(O.mx_pack(q), s)
    x, xv = rows(rng, M, K, kind, 2.0 ** xe)
    ref = xv @ wv.T
    lost = 2.0 ** -134 * np.abs(wv).sum(1) if kind == "f32" else 0.0
    check(_gemm(x, upload(q, s), N, kind), ref, out_bound(ref, gemm_bound(xv, wv, kind) + lost, torch.float32), kind)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_quantised_rows_and_weights_that_were_not_finite(M):
    """What the quantisers make of them (codes 0, scale byte 255) is NaN in every product, and alone."""
    rng = np.random.default_rng(M)
    K, N = 288, 112
    a, b = torch.as_tensor(rng.standard_normal((M, K))).float().cuda(), torch.as_tensor(rng.standard_normal((K, N))).float().cuda()
    b[77, 9] = float("inf")
    w = L.mx_quantize_to_weight(b)
    c = a.clone()
    c[2, 130], c[0, 5] = float("nan"), -float("inf")
    m = L.mx_empty(M, K)
    L.mx_quantize(c, m)
    for x, bad_rows in ((a, []), (a.bfloat16(), []), (m, [0, 2])):
        nan = _gemm(x, w, N, "mx" if x is m else "f32" if x.dtype == torch.float32 else "bf16").isnan().cpu()
        want = torch.zeros((M, N), dtype=torch.bool)
        want[:, 9], want[bad_rows] = True, True
        assert torch.equal(nan, want)


def test_weights_made_on_another_stream_and_freed_while_in_use():
    """Their memory is that stream's: the next weights made there are not put over them before the current
    stream's product, still waiting behind other work, has read them."""
    torch.manual_seed(5)
    a, b = torch.randn((4096, 4096), device="cuda"), torch.randn((4096, 4096), device="cuda")
    x, busy = torch.randn((4, 4096), device="cuda"), torch.randn((4096, 4096), device="cuda")
    want = _gemm(x, L.mx_quantize_to_weight(a), 4096, "f32")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ws = L.new_workspace(L.mx_gemm_workspace_bytes(4, L.F32, L.mx_quantize_to_weight(a)))
    y = torch.empty_like(want)
    w = L.mx_quantize_to_weight(a, side)
    torch.cuda.synchronize()
    for _ in range(40):
        torch.mm(busy, busy, out=b)  # some 40 ms
    L.mx_gemm(x, w, y, ws)
    del w
    other = [L.mx_quantize_to_weight(busy, side) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and len(other) == 3
