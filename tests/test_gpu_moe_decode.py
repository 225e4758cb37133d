"""GPU parity of w4a16_moe_decode against the float64 oracle (router and layer),
element by element, and its agreement with the calls it stands in for."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
import workloads as W
from helpers import rel_err, tol_for, weight_from_codes, x_for_dtype, x_values
from lora_bounds import HALF_STEP, codes
from oracle_pool import TAU, ExpertPool, check_elementwise, mlp_bound, moe_bound_from

pytestmark = pytest.mark.gpu

TYPES = [("f32", torch.float32), ("bf16", torch.bfloat16), ("bf16", torch.float32), ("f32", torch.bfloat16)]


def _stacks(E, H, I, seed, group=32):
    """Per projection (codes [E][K/8][N], scales), on the host."""
    out = []
    for i, (K, N) in enumerate(((H, I), (H, I), (I, H))):
        qs, ss = zip(*(codes(K, N, seed + 1000 * i + e, group) for e in range(E)))
        out.append((np.stack(qs), np.stack(ss)))
    return out


def _device(stacks):
    return [weight_from_codes(*s) for s in stacks]


def _run(x, logits, k, ws3, ytype, shared=None, ws=None, out=True, stream=None):
    M, E = logits.shape
    buf = torch.full((M + 2, ws3[2].N), 7.0, dtype=ytype, device="cuda")
    ids = torch.full((M + 1, k), -7, dtype=torch.int32, device="cuda") if out else None
    w = torch.full((M + 1, k), -7.0, device="cuda") if out else None
    if ws is None:
        ws = L.new_workspace(L.moe_decode_workspace_bytes(M, k, L._dtype_code(x), *ws3, shared=shared))
    L.moe_decode(x, logits, k, *ws3, buf[:M], ws, shared, ids[:M] if out else None, w[:M] if out else None, stream)
    torch.cuda.synchronize()
    assert bool((buf[M:] == 7.0).all()), "rows behind the last were written"
    if out:
        assert bool((ids[M:] == -7).all()) and bool((w[M:] == -7.0).all())
        return buf[:M], ids[:M], w[:M]
    return buf[:M]


def _reference(xv, ids, w, stacks, shared, dtype, ytype):
    E = stacks[0][0].shape[0]

    def expert(e):
        return tuple((q[e], s[e]) for q, s in stacks)

    with ExpertPool(TAU[dtype], workers=0) as pool:
        if shared is None:
            ref = O.moe64(xv, ids, w, expert, E, map_fn=pool)
        else:
            one = tuple((q[0], s[0]) for q, s in shared)
            ref = O.moe_shared64(xv, ids, w, expert, E, one, map_fn=pool)
        bound = moe_bound_from(pool.bounds, ids, w)
    if shared is not None:
        bound = bound + mlp_bound(xv, *one, TAU[dtype])
    return ref, bound + HALF_STEP[ytype] * (np.abs(ref) + bound)


def _check_layer(M, H, I, E, k, dtype, ytype, seed, shared=False, group=32, logits=None):
    stacks = _stacks(E, H, I, seed, group)
    sh = _stacks(1, H, I, seed + 7, group) if shared else None
    x = x_for_dtype(W.activations(M, H, seed), dtype).cuda()
    lg = W.router_logits(M, E, seed) if logits is None else logits
    y, ids, w = _run(x, lg.cuda(), k, _device(stacks), ytype, _device(sh) if shared else None)
    want_ids, want_w = O.moe_topk(lg.numpy(), k)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=1e-6, atol=1e-30)
    ref, bound = _reference(x_values(x), want_ids, want_w, stacks, sh, dtype, ytype)
    what = f"moe_decode M={M} H={H} I={I} E={E} k={k} {dtype}->{ytype} shared={shared} group={group}"
    worst = check_elementwise(y.double().cpu().numpy(), ref, bound, what)
    err = rel_err(y.double(), ref)
    print(f"{what} relF={err:.3e} worst/bound={worst:.2e}", flush=True)
    if ytype == torch.float32:
        assert err <= tol_for(dtype)


@pytest.mark.parametrize("dtype,ytype", TYPES)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("H,I,E,k", [(64, 64, 1, 1), (64, 64, 6, 2), (256, 128, 4, 4), (512, 192, 20, 3),
                                     (1024, 320, 9, 8), (128, 704, 65, 5)])
@pytest.mark.parametrize("M", [1, 3, 8, 11, 16])
def test_layers(M, H, I, E, k, shared, dtype, ytype):
    if dtype == "f32" and M > 8:
        M -= 8
    _check_layer(M, H, I, E, k, dtype, ytype, 300 + M, shared)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,H,I,E,k", [
    (16, 256, 704, 130, 8),   # more work items than a round of workgroups: one quad, no K split
    (16, 2560, 64, 70, 8),    # several windows of one quad; down: many experts of two groups each
    (1, 2560, 192, 4, 2),     # four quads and K splits
    (4, 2048, 448, 24, 8),
    (2, 4096, 64, 3, 3),
    (5, 128, 2048, 8, 2),     # a long intermediate: windows inside one expert
    (7, 64, 64, 1024, 32),    # the largest router
    (8, 64, 128, 300, 32),
])
def test_launch_shapes(M, H, I, E, k, dtype):
    _check_layer(min(M, 8 if dtype == "f32" else 16), H, I, E, k, dtype, torch.float32, 400 + M, shared=M % 2 == 0)


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_group_sizes(group, dtype):
    _check_layer(6, 640, 384, 12, 3, dtype, torch.float32, 500, True, group)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 8, 16])
def test_every_token_picks_the_same_experts(M, dtype):
    M = min(M, 8 if dtype == "f32" else 16)
    lg = torch.zeros((M, 30))
    lg[:, 7], lg[:, 29] = 2.0, 1.0
    _check_layer(M, 256, 192, 30, 2, dtype, torch.float32, 520, logits=lg)


@pytest.mark.parametrize("E,k", [(6, 6), (64, 8), (65, 9), (129, 8), (384, 8), (513, 32), (1024, 5)])
def test_choice_is_that_of_moe_topk(E, k):
    """Integer logits (many ties), bit for bit."""
    lg = torch.from_numpy(np.random.default_rng(E).integers(-3, 3, (8, E)).astype(np.float32)).cuda()
    lg[3] *= 1e38
    lg[4] = -0.0
    lg[4, ::2] = 0.0
    lg[5] = torch.randn(E, generator=torch.Generator().manual_seed(1)).cuda()
    ws3 = _device(_stacks(1, 64, 64, 530))
    ws3 = [L.Weight(w.qw.expand(E, *w.qw.shape[1:]).contiguous(), w.scales.expand(E, *w.scales.shape[1:]).contiguous(),
                    w.K, w.N, E) for w in ws3]
    x = torch.randn((8, 64), generator=torch.Generator().manual_seed(2)).cuda()
    _, ids, w = _run(x, lg, k, ws3, torch.float32)
    want_ids, want_w = torch.empty_like(ids), torch.empty_like(w)
    L.moe_topk(lg, k, want_ids, want_w)
    torch.cuda.synchronize()
    assert torch.equal(ids, want_ids)
    assert torch.equal(w, want_w)


def test_logits_that_are_not_finite():
    """NaN counts as -infinity, +infinity as the largest float; a token with nothing
    above -infinity takes the shared expert alone, and its rows read no expert."""
    H, I, E, k = 128, 64, 8, 3
    inf, nan, big = float("inf"), float("nan"), float(np.finfo(np.float32).max)
    rows = [[-inf] * 8, [nan] * 8, [-inf, 1.0, nan, -inf, -inf, 0.0, -inf, -inf], [inf, 0, inf, 1, 2, 3, 4, 5],
            [0, 1, big, inf, -inf, nan, -big, 2], [-big] * 8, [-inf, -inf, -inf, -inf, -inf, -inf, -inf, 3.0]]
    lg = torch.tensor(rows, dtype=torch.float32)
    clean = np.clip(np.where(np.isnan(lg.numpy()), -np.inf, lg.numpy()), -np.inf, big).astype(np.float64)
    # selection by the values before +infinity is clamped
    order = np.where(np.isnan(lg.numpy()), -np.inf, lg.numpy())
    want_ids = np.array([sorted(range(E), key=lambda e: (-r[e], e))[:k] for r in order], np.int32)
    v = np.take_along_axis(clean, want_ids.astype(np.int64), 1)
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.where(v[:, :1] > -np.inf, np.exp(v - v[:, :1]), 0.0)
    want_w = z / np.maximum(z.sum(1, keepdims=True), 1e-300)
    stacks, sh = _stacks(E, H, I, 540), _stacks(1, H, I, 541)
    # an expert whose weight is 0 for every token holds infinities
    unread = sorted(set(range(E)) - {int(e) for t in range(len(rows)) for e, p in zip(want_ids[t], want_w[t]) if p > 0})
    assert unread
    dev = [(q, s.copy()) for q, s in stacks]
    for _, s in dev:
        s[unread] = np.inf
    M = len(rows)
    x = W.activations(M, H, 542).cuda()
    for shared in (None, sh):
        y, ids, w = _run(x, lg.cuda(), k, _device(dev), torch.float32, None if shared is None else _device(shared))
        np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
        np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=1e-6)
        ref, bound = _reference(x_values(x), want_ids, want_w, stacks, shared, "f32", torch.float32)
        check_elementwise(y.cpu().numpy(), ref, bound, "moe_decode with masked experts")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_bad_row_stays_its_own(dtype):
    H, I, E, k, M = 256, 128, 6, 3, 8
    ws3 = _device(_stacks(E, H, I, 550))
    x = x_for_dtype(W.activations(M, H, 551), dtype).cuda()
    lg = W.router_logits(M, E, 552).cuda()
    want = _run(x, lg, k, ws3, torch.float32, out=False)
    for bad in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[2, 5] = bad
        got = _run(x2, lg, k, ws3, torch.float32, out=False)
        keep = torch.arange(M, device="cuda") != 2
        assert torch.equal(got[keep], want[keep])
        assert not bool(torch.isfinite(got[2]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 5, 8])
@pytest.mark.parametrize("shared", [False, True])
def test_replays_streams_and_one_workspace(M, shared, dtype):
    """The same bits from repeated calls on one workspace with other tokens between, from
    a replayed graph whose logits change, and on a side stream."""
    H, I, E, k = 512, 192, 24, 4
    ws3 = _device(_stacks(E, H, I, 560))
    sh = _device(_stacks(1, H, I, 561)) if shared else None
    x = x_for_dtype(W.activations(M, H, 562), dtype).cuda()
    lgs = [W.router_logits(M, E, 563 + i).cuda() for i in range(3)]
    lgs[2][:] = -float("inf")  # nothing chosen
    want = [_run(x, lg, k, ws3, torch.float32, sh) for lg in lgs]
    nbytes = L.moe_decode_workspace_bytes(M, k, L._dtype_code(x), *ws3, shared=sh)
    ws, gws = L.new_workspace(nbytes), L.new_workspace(nbytes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for ref, lg in zip(want, lgs):
        for st in (None, side):
            got = _run(x, lg, k, ws3, torch.float32, sh, ws, stream=st)
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
    cur, y = lgs[0].clone(), torch.empty((M, H), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.moe_decode(x, cur, k, *ws3, y, gws, sh)
    for ref, lg in list(zip(want, lgs)) * 2:
        cur.copy_(lg)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref[0])
        assert torch.equal(_run(x, lg, k, ws3, torch.float32, sh, ws)[0], ref[0])


def test_m0_writes_nothing():
    ws3 = _device(_stacks(3, 64, 64, 570))
    L.moe_decode(torch.empty((0, 64), device="cuda"), torch.empty((0, 3), device="cuda"), 2, *ws3,
                 torch.empty((0, 64), device="cuda"), L.new_workspace(256))
    torch.cuda.synchronize()
