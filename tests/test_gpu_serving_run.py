"""The adapter projections and the few-token MoE layer as they are served: one decode
step of both in a row (eager and replayed), sizes that take their other launch shapes,
stacks past 32-bit offsets, and two streams at once."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
import workloads as W
from helpers import x_for_dtype, x_values
from lora_bounds import (HALF_STEP, adapters, codes, device_lora, device_weight, gemm_lora_bound, id_pattern,
                         mlp_lora_bound)
from oracle_pool import TAU, ExpertPool, check_elementwise, moe_bound_from
from test_gpu_lora import TYPES, _check, _code, _gemm, _mlp, _x
from test_gpu_moe_decode import _device, _reference, _run, _stacks

pytestmark = pytest.mark.gpu


class Step:
    """A projection with adapters, an MLP with adapters, the MoE layer, on one workspace
    and without a host step between; the residual sums are torch's."""

    def __init__(self, M, dtype, seed):
        self.M, self.dtype, self.k = M, dtype, 4
        H, I, E, n = 512, 384, 24, 5
        self.w = [codes(H, H, seed), codes(H, I, seed + 1), codes(H, I, seed + 2), codes(I, H, seed + 3)]
        self.lo = [adapters(n, 16, H, H, seed + 4), adapters(n, 8, H, I, seed + 5), None,
                   adapters(n, 24, I, H, seed + 6, ranks=[24, 3, 0, 8, 17])]
        self.stacks, self.shared = _stacks(E, H, I, seed + 7), _stacks(1, H, I, seed + 8)
        self.dw, self.dlo = [device_weight(w) for w in self.w], [device_lora(l) for l in self.lo]
        self.ds, self.dsh = _device(self.stacks), _device(self.shared)
        code = _code(dtype)
        need = max(L.gemm_lora_workspace_bytes(M, self.dw[0], code, self.dlo[0]),
                   L.swiglu_mlp_lora_workspace_bytes(M, code, *self.dw[1:], *self.dlo[1:]),
                   L.moe_decode_workspace_bytes(M, self.k, code, *self.ds, shared=self.dsh))
        self.need = need
        self.outs = [torch.empty((M, H), device="cuda") for _ in range(3)]
        self.xs = [None, None]

    def run(self, x, ids, logits, ws):
        t = x.dtype
        L.gemm_lora(x, self.dw[0], self.dlo[0], ids, self.outs[0], ws)
        x1 = (x.float() + self.outs[0]).to(t)
        L.swiglu_mlp_lora(x1, *self.dw[1:], *self.dlo[1:], ids, self.outs[1], ws)
        x2 = (x1.float() + self.outs[1]).to(t)
        L.moe_decode(x2, logits, self.k, *self.ds, self.outs[2], ws, self.dsh)
        self.xs = [x1, x2]

    def check(self, x, ids, logits):
        """Each operator's output against the oracle of what went into it."""
        d, f32 = self.dtype, torch.float32
        idh = ids.cpu().numpy()
        xv, x1, x2 = (x_values(t.cpu()) for t in (x, *self.xs))
        got = [o.double().cpu().numpy() for o in self.outs]
        check_elementwise(got[0], O.gemm_lora64(xv, self.w[0], self.lo[0], idh),
                          gemm_lora_bound(xv, self.w[0], self.lo[0], idh, d, f32), "projection")
        check_elementwise(got[1], O.swiglu_mlp_lora64(x1, *self.w[1:], *self.lo[1:], idh),
                          mlp_lora_bound(x1, *self.w[1:], *self.lo[1:], idh, d, f32), "mlp")
        ci, cw = O.moe_topk(logits.cpu().numpy(), self.k)
        ref, bound = _reference(x2, ci, cw, self.stacks, self.shared, d, f32)
        check_elementwise(got[2], ref, bound, "moe")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 4, 8, 16])
def test_a_decode_step(M, dtype):
    M = min(M, 8 if dtype == "f32" else 16)
    step = Step(M, dtype, 900 + M)
    ws, gws = L.new_workspace(step.need), L.new_workspace(step.need)
    xs = [_x(M, 512, dtype, 910 + i) for i in range(2)]
    idv = [torch.from_numpy(id_pattern(k, M, 5, 920)).cuda() for k in ("random", "distinct")]
    lgs = [W.router_logits(M, 24, 930 + i).cuda() for i in range(2)]
    want = []
    for a in zip(xs, idv, lgs):
        step.run(*a, ws)
        torch.cuda.synchronize()
        step.check(*a)
        want.append([o.clone() for o in step.outs])
    cur = [xs[0].clone(), idv[0].clone(), lgs[0].clone()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(*cur, gws)
    for i in (0, 1, 1, 0, 1):
        for dst, src in zip(cur, (xs[i], idv[i], lgs[i])):
            dst.copy_(src)
        for o in step.outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step.outs, want[i]))
        step.run(xs[1 - i], idv[1 - i], lgs[1 - i], ws)  # the program's own calls between
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step.outs, want[1 - i]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_streams_at_once(dtype):
    """Calls in flight together on streams and workspaces of their own give the bits of
    calls one after another."""
    M = 8
    steps = [Step(M, dtype, 940), Step(M, dtype, 941)]
    x = [_x(M, 512, dtype, 942 + i) for i in range(2)]
    ids = [torch.from_numpy(id_pattern("random", M, 5, 944 + i)).cuda() for i in range(2)]
    lg = [W.router_logits(M, 24, 946 + i).cuda() for i in range(2)]
    ws = [L.new_workspace(s.need) for s in steps]
    want = []
    for i in range(2):
        steps[i].run(x[i], ids[i], lg[i], ws[i])
        torch.cuda.synchronize()
        want.append([o.clone() for o in steps[i].outs])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            for o in steps[i].outs:
                o.fill_(float("nan"))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                steps[i].run(x[i], ids[i], lg[i], ws[i])
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(steps[i].outs, want[i]))


@pytest.mark.parametrize("dtype,ytype", TYPES)
@pytest.mark.parametrize("K,N,R,n", [(4064, 192, 16, 7), (8192, 64, 8, 3), (96, 1024, 256, 2), (1600, 704, 40, 64)])
@pytest.mark.parametrize("M", [10, 18, 31, 32, 33, 47, 49, 63])
def test_gemm_lora_up_to_64_rows(M, K, N, R, n, dtype, ytype):
    """K that does not divide into the parts and splits, one column block, more columns
    than a workgroup's."""
    w, lo = codes(K, N, K + N), adapters(n, R, K, N, R)
    ids = id_pattern("random", M, n, M)
    x = _x(M, K, dtype, 60 + M)
    y = _gemm(x, device_weight(w), device_lora(lo), torch.from_numpy(ids).cuda(), ytype)
    xv = x_values(x)
    _check(y, O.gemm_lora64(xv, w, lo, ids), gemm_lora_bound(xv, w, lo, ids, dtype, ytype),
           f"gemm_lora M={M} K={K} N={N} R={R} n={n} {dtype}->{ytype}", dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,I", [(320, 448), (1088, 64), (64, 2048)])
@pytest.mark.parametrize("M", [12, 20, 48, 50])
def test_mlp_lora_up_to_64_rows(M, H, I, dtype):
    shapes = [(H, I), (H, I), (I, H)]
    ws3 = [codes(K, N, 70 + i) for i, (K, N) in enumerate(shapes)]
    los = [adapters(4, 16, K, N, 73 + i) for i, (K, N) in enumerate(shapes)]
    ids = id_pattern("random", M, 4, 76)
    x = _x(M, H, dtype, 77)
    y = _mlp(x, [device_weight(w) for w in ws3], [device_lora(l) for l in los], torch.from_numpy(ids).cuda(),
             torch.float32)
    xv = x_values(x)
    _check(y, O.swiglu_mlp_lora64(xv, *ws3, *los, ids), mlp_lora_bound(xv, *ws3, *los, ids, dtype, torch.float32),
           f"mlp_lora M={M} H={H} I={I} {dtype}", dtype)


@pytest.mark.parametrize("dtype,ytype", TYPES)
@pytest.mark.parametrize("M,K,N,R,n,kind", [
    (1100, 128, 4096, 24, 5, "segments"),   # tall blocks of the finish
    (1100, 192, 4096, 8, 3, "random"),      # K without wide tiles
    (512, 256, 256, 32, 40, "random"),      # the largest by rows, and one row more
    (513, 256, 256, 32, 40, "random"),
    (600, 384, 64, 200, 9, "segments"),     # several chunks of ranks
])
def test_gemm_lora_many_rows(M, K, N, R, n, kind, dtype, ytype):
    w, lo = codes(K, N, K + N), adapters(n, R, K, N, R, ranks=[(7 * i) % (R + 1) for i in range(n)])
    ids = id_pattern(kind, M, n, M)
    x = _x(M, K, dtype, 80)
    y = _gemm(x, device_weight(w), device_lora(lo), torch.from_numpy(ids).cuda(), ytype)
    xv = x_values(x)
    _check(y, O.gemm_lora64(xv, w, lo, ids), gemm_lora_bound(xv, w, lo, ids, dtype, ytype),
           f"gemm_lora M={M} K={K} N={N} R={R} n={n} {kind} {dtype}->{ytype}", dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mlp_lora_many_rows(dtype):
    M, H, I = 1030, 128, 4096
    shapes = [(H, I), (H, I), (I, H)]
    ws3 = [codes(K, N, 84 + i) for i, (K, N) in enumerate(shapes)]
    los = [adapters(4, 24, K, N, 87 + i) for i, (K, N) in enumerate(shapes)]
    ids = id_pattern("segments", M, 4, 90)
    x = _x(M, H, dtype, 91)
    y = _mlp(x, [device_weight(w) for w in ws3], [device_lora(l) for l in los], torch.from_numpy(ids).cuda(),
             torch.bfloat16)
    xv = x_values(x)
    _check(y, O.swiglu_mlp_lora64(xv, *ws3, *los, ids), mlp_lora_bound(xv, *ws3, *los, ids, dtype, torch.bfloat16),
           f"mlp_lora M={M} H={H} I={I} {dtype}", dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_few_rows_of_a_very_long_k(dtype):
    """Windows of all the splits together hold less than K: the tiles take it."""
    M, K, N = (8 if dtype == "f32" else 16), 33 * 8192, 64
    w, lo = codes(K, N, 92), adapters(2, 8, K, N, 93)
    ids = id_pattern("random", M, 2, 94)
    x = _x(M, K, dtype, 95)
    y = _gemm(x, device_weight(w), device_lora(lo), torch.from_numpy(ids).cuda(), torch.float32)
    xv = x_values(x)
    _check(y, O.gemm_lora64(xv, w, lo, ids), gemm_lora_bound(xv, w, lo, ids, dtype, torch.float32),
           f"gemm_lora M={M} K={K} {dtype}", dtype)


@pytest.mark.parametrize("M", [3, 40, 600])
@pytest.mark.parametrize("K,N", [(8192, 64), (64, 8192)])
def test_adapter_stacks_past_32_bit_offsets(M, K, N):
    """4.4 GB of a or of b; the last adapters are the ones in use."""
    R, n, used = 64, 4200, 3
    w, lo = codes(K, N, 96), adapters(used, R, K, N, 97)
    small = device_lora(lo)
    big = L.Lora(torch.zeros((n, R, K), dtype=torch.bfloat16, device="cuda"),
                 torch.zeros((n, N, R), dtype=torch.bfloat16, device="cuda"), torch.zeros(n, device="cuda"))
    for b, s in zip((big.a, big.b, big.scale), (small.a, small.b, small.scale)):
        b[n - used:] = s
    ids = id_pattern("distinct", M, used, 0)
    x = _x(M, K, "bf16", 98)
    dw = device_weight(w)
    y = _gemm(x, dw, big, torch.from_numpy(ids + n - used).cuda(), torch.float32)
    xv = x_values(x)
    _check(y, O.gemm_lora64(xv, w, lo, ids), gemm_lora_bound(xv, w, lo, ids, "bf16", torch.float32),
           f"gemm_lora M={M} K={K} N={N} n={n}", "bf16")
    assert torch.equal(y, _gemm(x, dw, small, torch.from_numpy(ids).cuda(), torch.float32))


@pytest.mark.parametrize("M", [1, 6])
def test_expert_stacks_past_32_bit_offsets(M):
    """1000 experts of 4.2 MB codes a projection; the first and the last ones are chosen."""
    H, I, E, k, used = 2048, 4096, 1000, 3, [0, 1, 997, 998, 999]
    host = _stacks(len(used), H, I, 99)
    ws3 = []
    for (K, N), small in zip(((H, I), (H, I), (I, H)), _device(host)):
        qw = torch.zeros((E, K // 32, N // 64, 64, 4), dtype=torch.int32, device="cuda")
        sc = torch.zeros((E, K // 32, N), device="cuda")
        for i, e in enumerate(used):
            qw[e] = small.qw.reshape(len(used), K // 32, N // 64, 64, 4)[i]
            sc[e] = small.scales[i]
        ws3.append(L.Weight(qw, sc, K, N, E))
    rng = np.random.default_rng(5)
    lg = torch.full((M, E), -50.0)
    lg[:, used] = torch.from_numpy(rng.standard_normal((M, len(used))).astype(np.float32))
    x = x_for_dtype(W.activations(M, H, 100), "f32").cuda()
    y, ids, w = _run(x, lg.cuda(), k, ws3, torch.float32)
    want_ids, want_w = O.moe_topk(lg.numpy(), k)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    place = {e: i for i, e in enumerate(used)}

    def expert(e):
        return tuple((q[place[e]], s[place[e]]) for q, s in host)

    with ExpertPool(TAU["f32"], workers=0) as pool:
        ref = O.moe64(x_values(x), want_ids, want_w, expert, E, map_fn=pool)
        bound = moe_bound_from(pool.bounds, want_ids, want_w)
    bound = bound + HALF_STEP[torch.float32] * (np.abs(ref) + bound)
    check_elementwise(y.double().cpu().numpy(), ref, bound, f"moe_decode E={E} M={M}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,H,I,kind", [
    (300, 1024, 1024, "random"),     # bf16: wide tiles that split K, gate and up one after the other
    (600, 2048, 512, "segments"),    # the same before the finish by blocks
    (180, 512, 4096, "random"),      # 64-row tiles: gate and up in a launch each
    (70, 2048, 1024, "random"),      # and in one
    (520, 1088, 704, "segments"),    # K the wide tiles do not take
])
def test_mlp_lora_launch_shapes_and_one_workspace(M, H, I, kind, dtype):
    """The base products' launch shapes; repeated calls on one workspace give the same bits."""
    shapes = [(H, I), (H, I), (I, H)]
    ws3 = [codes(K, N, 101 + i) for i, (K, N) in enumerate(shapes)]
    los = [adapters(6, 16, K, N, 104 + i) for i, (K, N) in enumerate(shapes)]
    ids = id_pattern(kind, M, 6, 107)
    x = _x(M, H, dtype, 108)
    dw, dlo, di = [device_weight(w) for w in ws3], [device_lora(l) for l in los], torch.from_numpy(ids).cuda()
    ws = L.new_workspace(L.swiglu_mlp_lora_workspace_bytes(M, _code(dtype), *dw, *dlo))
    first = _mlp(x, dw, dlo, di, torch.float32, ws)
    xv = x_values(x)
    _check(first, O.swiglu_mlp_lora64(xv, *ws3, *los, ids), mlp_lora_bound(xv, *ws3, *los, ids, dtype, torch.float32),
           f"mlp_lora M={M} H={H} I={I} {dtype}", dtype)
    for _ in range(3):
        assert torch.equal(_mlp(x, dw, dlo, di, torch.float32, ws), first)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", [(300, 4096, 256), (600, 2048, 512), (80, 4096, 128), (1100, 1024, 1024)])
def test_gemm_lora_launch_shapes_and_one_workspace(M, K, N, dtype):
    """Base products that split K, by rows and by blocks of the finish."""
    w, lo = codes(K, N, 111), adapters(6, 16, K, N, 112)
    ids = id_pattern("random", M, 6, 113)
    x = _x(M, K, dtype, 114)
    dw, dlo, di = device_weight(w), device_lora(lo), torch.from_numpy(ids).cuda()
    ws = L.new_workspace(L.gemm_lora_workspace_bytes(M, dw, _code(dtype), dlo))
    first = _gemm(x, dw, dlo, di, torch.float32, ws)
    xv = x_values(x)
    _check(first, O.gemm_lora64(xv, w, lo, ids), gemm_lora_bound(xv, w, lo, ids, dtype, torch.float32),
           f"gemm_lora M={M} K={K} N={N} {dtype}", dtype)
    for _ in range(3):
        assert torch.equal(_gemm(x, dw, dlo, di, torch.float32, ws), first)
