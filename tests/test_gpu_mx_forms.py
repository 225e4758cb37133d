"""MXFP4 products in the forms that test_gpu_mx.py's shapes no longer reach since more of them are
streamed: h handed from one form to another, shared tiles on two streams.  Every form is asserted
(mx_plan.py), so a change of the rule shows here."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import mx_plan
import oracle as O
from mx_bounds import big_weight, check, code_of, gemm_bound, mlp_reference, out_bound, rows, upload

pytestmark = pytest.mark.gpu

# (kind, M, H, I, gate and up's form, down's)
MLPS = [
    ("f32", 17, 64, 18464, "stream", "32x256 shared"), ("f32", 33, 64, 32992, "stream", "64x256 shared"),
    ("f32", 65, 64, 32992, "stream", "128x256 shared"), ("f32", 20, 2080, 18464, "32x128", "32x256 shared"),
    ("f32", 17, 4128, 7200, "32x128 shared", "32x256 shared"), ("f32", 17, 7168, 2080, "32x128 shared", "stream"),
    ("f32", 50, 256, 32992, "64x128", "64x256 shared"), ("f32", 50, 2080, 9248, "64x128 shared", "64x256 shared"),
    ("f32", 50, 7168, 2080, "64x128 shared", "stream"), ("f32", 100, 256, 18464, "128x128", "stream"),
    ("f32", 100, 4128, 4128, "128x128 shared", "stream"), ("f32", 150, 64, 544, "128x128", "128x256 shared"),
    ("f32", 150, 544, 64, "128x128 shared", "128x256"), ("f32", 150, 544, 544, "128x128 shared", "128x256 shared"),
    ("f32", 150, 544, 18464, "128x128 rest 64x128", "128x256 shared"),
    ("bf16", 17, 64, 18464, "stream", "32x256 shared"), ("bf16", 33, 64, 18464, "stream", "64x256 shared"),
    ("bf16", 65, 64, 32992, "stream", "128x256 shared"), ("bf16", 17, 544, 32992, "32x128", "32x256 shared"),
    ("bf16", 17, 4128, 4128, "32x128 shared", "32x256 shared"), ("bf16", 17, 7168, 64, "32x128 shared", "stream"),
    ("bf16", 50, 256, 32992, "64x128", "64x256 shared"), ("bf16", 50, 2080, 7200, "64x128 shared", "64x256 shared"),
    ("bf16", 33, 4128, 4128, "64x128 shared", "stream"), ("bf16", 100, 256, 18464, "128x128", "stream"),
    ("bf16", 128, 7168, 1056, "128x128 shared", "stream"), ("bf16", 150, 1056, 64, "128x128 shared", "128x256"),
    ("bf16", 150, 1056, 544, "128x128 shared", "128x256 shared"),
    ("mx", 17, 64, 18464, "stream", "32x256 shared"), ("mx", 33, 64, 18464, "stream", "64x256 shared"),
    ("mx", 65, 64, 18464, "stream", "128x256 shared"), ("mx", 17, 256, 32992, "32x128", "32x256 shared"),
    ("mx", 17, 2080, 9248, "32x128 shared", "32x256 shared"), ("mx", 17, 7168, 64, "32x128 shared", "stream"),
    ("mx", 50, 64, 32992, "64x128", "64x256 shared"), ("mx", 50, 1056, 9248, "64x128", "stream"),
    ("mx", 50, 4128, 4128, "64x128 shared", "64x256 shared"), ("mx", 33, 7168, 64, "64x128 shared", "stream"),
    ("mx", 100, 256, 9248, "128x128", "stream"), ("mx", 65, 7168, 64, "128x128 shared", "stream"),
    ("mx", 150, 64, 18464, "128x256", "128x256 shared"), ("mx", 150, 2080, 2080, "128x128 shared", "128x256 shared"),
]


def _assert_forms(M, H, I, kind, gu, dn):
    assert tuple(map(str, mx_plan.mlp(M, H, I, kind))) == (gu, dn)


@pytest.mark.parametrize("kind,M,H,I,gu,dn", MLPS)
def test_mlp_hands_h_from_form_to_form(kind, M, H, I, gu, dn):
    _assert_forms(M, H, I, kind, gu, dn)
    rng = np.random.default_rng(M + H + I)
    (g, gv), (u, uv), (d, dv) = big_weight(rng, I, H, 0.06), big_weight(rng, I, H, 0.06), big_weight(rng, H, I, 0.06)
    x, xv = rows(rng, M, H, kind)
    y = torch.full((M + 1, H), 7.0, device="cuda")
    size = L.mx_swiglu_mlp_workspace_bytes(M, code_of(kind), g, u, d)
    assert size == mx_plan.mlp_bytes(M, H, I, kind)
    ws = L.new_workspace(size)
    L.mx_swiglu_mlp(x, g, u, d, y[:M], ws)
    ref, b = mlp_reference(xv, gv, uv, dv, kind)
    check(y[:M], ref, out_bound(ref, b, torch.float32), f"{M}x{H}x{I} {kind}")
    assert y[M].eq(7.0).all()
    again = torch.empty((M, H), device="cuda")
    L.mx_swiglu_mlp(x, g, u, d, again, ws)
    assert torch.equal(y[:M], again)


def _one_hot(N, K, at, code):
    q = np.zeros((N, K), np.uint8)
    q[np.arange(N), at] = code
    return upload(q, np.full((N, K // 32), 127, np.uint8))


@pytest.mark.parametrize("kind,M,H,I,gu,dn", [c for c in MLPS if c[0] == "f32"])
def test_float32_h_keeps_every_bit(kind, M, H, I, gu, dn):
    """gate = 32 (its silu is 32), up one value of 24 bits a row, down half of one column of h: exact."""
    _assert_forms(M, H, I, kind, gu, dn)
    rng = np.random.default_rng(M + H + I)
    x = np.zeros((M, H), np.float32)
    v = np.ldexp((rng.integers(1 << 22, 1 << 23, M) * 2 + 1).astype(np.float64), -23)
    x[:, 0], x[:, H - 1] = 16.0, v
    g, u = _one_hot(I, H, np.zeros(I, int), 4), _one_hot(I, H, np.full(I, H - 1), 2)  # 2 x[0], 1 x[H - 1]
    d = _one_hot(H, I, rng.integers(0, I, H), 1)
    y = torch.empty((M, H), device="cuda")
    L.mx_swiglu_mlp(torch.as_tensor(x).cuda(), g, u, d, y, L.new_workspace(L.mx_swiglu_mlp_workspace_bytes(M, L.F32, g, u, d)))
    assert torch.equal(y.cpu(), torch.as_tensor(np.repeat(16 * v[:, None], H, 1).astype(np.float32)))


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("M,K,N", [(64, 7136, 4112), (17, 7136, 4112), (150, 2336, 784)])
def test_shared_tiles_on_two_streams(M, K, N, kind):
    """Each call's sums lie in its own workspace; the same bits as one after the other."""
    assert mx_plan.product(M, N, K, kind).plane_bytes >= 2 * M * N * 4
    rng = np.random.default_rng(M + K)
    w, wv = big_weight(rng, N, K)
    xs = [rows(rng, M, K, kind) for _ in range(2)]
    n = L.mx_gemm_workspace_bytes(M, code_of(kind), w)
    assert n == mx_plan.gemm_bytes(M, K, N, kind)
    wss, ys, want = [L.new_workspace(n) for _ in xs], [torch.empty((M, N), device="cuda") for _ in xs], []
    for x, xv in xs:
        want.append(torch.empty((M, N), device="cuda"))
        L.mx_gemm(x, w, want[-1], wss[0])
        ref = xv @ wv.T
        check(want[-1], ref, out_bound(ref, gemm_bound(xv, wv, kind), torch.float32), kind)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (x, _), y, ws in zip(streams, xs, ys, wss):
            L.mx_gemm(x, w, y, ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
def test_two_graphs_on_one_workspace(kind):
    """Captured calls that share a workspace, replayed in turn on one stream."""
    M, H, I = 50, 4128, 7200
    assert all(f.shared for f in mx_plan.mlp(M, H, I, kind))
    rng = np.random.default_rng(4)
    (g, _), (u, _), (d, _) = big_weight(rng, I, H), big_weight(rng, I, H), big_weight(rng, H, I)
    ws = L.new_workspace(L.mx_swiglu_mlp_workspace_bytes(M, code_of(kind), g, u, d))
    xs = [rows(rng, M, H, kind)[0] for _ in range(2)]
    ys, want, graphs = [torch.empty((M, H), device="cuda") for _ in xs], [], []
    for x, y in zip(xs, ys):
        L.mx_swiglu_mlp(x, g, u, d, y, ws)
        want.append(y.clone())
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            L.mx_swiglu_mlp(x, g, u, d, y, ws)
    for _ in range(3):
        ys[0].zero_(), ys[1].zero_()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])
