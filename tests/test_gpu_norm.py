"""block_norm on the GPU against float64.

float32 form: a mean of H squares is summed in at most 32 additions a thread and 6 + 16 more,
each half a step, so n's relative error is at most (54 / 2 + 8) 2^-24 < 2^-18 before its own
rounding; the residual adds as much of |alpha gate post(y)|.  n is checked from the stored s.
MXFP4 form: float64 throughout, so codes and scales are the oracle's bit for bit."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
from mx_bounds import HALF_STEP, TORCH, check

pytestmark = pytest.mark.gpu


def _f(t):
    return None if t is None else t.double().cpu().numpy()


def _inputs(rng, M, H, yt, rt, wt, post, gate):
    t = lambda ty, *s: torch.as_tensor(rng.standard_normal(s)).to(TORCH[ty]).cuda()  # noqa: E731
    return dict(y=t(yt, M, H), r=t(rt, M, H), pre_w=t(wt, H), post_w=t(wt, H) if post else None,
                gate={"none": None, "channel": t(wt, H), "row": t(wt, M, H)}[gate])


CASES = [
    (1, 8, "f32", "f32", "f32", True, "none"), (1, 7168, "bf16", "bf16", "bf16", True, "channel"),
    (4, 7168, "bf16", "f32", "f32", False, "row"), (3, 1000, "f32", "bf16", "bf16", True, "row"),
    (130, 256, "bf16", "bf16", "f32", True, "channel"), (33, 8200, "f32", "f32", "bf16", True, "row"),
    (5, 16392, "bf16", "bf16", "bf16", True, "channel"), (2, 32768, "f32", "f32", "f32", False, "none"),
    (1000, 96, "bf16", "f32", "bf16", False, "channel"),
    # more rows than workgroups: each takes several
    (600, 7168, "bf16", "bf16", "bf16", True, "row"), (1400, 2304, "bf16", "bf16", "bf16", False, "channel"),
    (530, 16384, "bf16", "bf16", "bf16", True, "none"), (4100, 64, "bf16", "bf16", "bf16", True, "channel"),
    (300, 7168, "f32", "f32", "f32", True, "row"),
]


@pytest.mark.parametrize("M,H,yt,rt,wt,post,gate", CASES)
def test_norm(M, H, yt, rt, wt, post, gate):
    a = _inputs(np.random.default_rng(M + H), M, H, yt, rt, wt, post, gate)
    for nt in ("f32", "bf16"):
        r_out = torch.full_like(a["r"], float("nan"))
        n = torch.full((M, H), float("nan"), dtype=TORCH[nt], device="cuda")
        L.block_norm(a["y"], a["r"], r_out, n, pre_w=a["pre_w"], post_w=a["post_w"], gate=a["gate"], alpha=0.75, eps=1e-5)
        s, _ = O.block_norm64(_f(a["y"]), _f(a["r"]), _f(a["post_w"]), _f(a["gate"]), 0.75, 1e-5)
        part = np.abs(s - _f(a["r"]))
        b = 2.0 ** -18 * part + 2.0 ** -23 * np.abs(s)
        check(r_out, s, b + HALF_STEP[r_out.dtype] * (np.abs(s) + b) + 1e-37, "residual")
        _, nv = O.block_norm64(_f(r_out), eps=1e-5, pre_w=_f(a["pre_w"]))
        check(n, nv, (2.0 ** -18 + HALF_STEP[n.dtype]) * np.abs(nv) + 1e-37, "norm")
    # in place, and the parts alone
    r, n2 = a["r"].clone(), torch.empty_like(n)
    L.block_norm(a["y"], r, r, n2, pre_w=a["pre_w"], post_w=a["post_w"], gate=a["gate"], alpha=0.75, eps=1e-5)
    assert torch.equal(r, r_out) and torch.equal(n2, n)
    n3 = torch.empty_like(n)
    L.block_norm(r_out, n=n3, pre_w=a["pre_w"], eps=1e-5)
    assert torch.equal(n3, n)
    r3 = torch.empty_like(r)
    L.block_norm(a["y"], a["r"], r3, post_w=a["post_w"], gate=a["gate"], alpha=0.75, eps=1e-5)
    assert torch.equal(r3, r_out)


@pytest.mark.parametrize("M,H,yt,rt,wt,post,gate", [c for c in CASES if c[1] % 32 == 0])
def test_norm_to_mxfp4_is_exact(M, H, yt, rt, wt, post, gate):
    a = _inputs(np.random.default_rng(M * H), M, H, yt, rt, wt, post, gate)
    r_out, n = torch.empty_like(a["r"]), L.mx_empty(M, H)
    L.block_norm(a["y"], a["r"], r_out, n, pre_w=a["pre_w"], post_w=a["post_w"], gate=a["gate"], alpha=0.75)
    stored = lambda s: torch.as_tensor(s).float().to(TORCH[rt]).double().numpy()  # noqa: E731
    s, nv = O.block_norm64(_f(a["y"]), _f(a["r"]), _f(a["post_w"]), _f(a["gate"]), 0.75, 1e-6, _f(a["pre_w"]), stored)
    assert np.array_equal(_f(r_out), stored(s))
    q, sc = O.mx_quantize64(nv)
    assert np.array_equal(n.scales.cpu().numpy(), sc) and np.array_equal(n.codes.cpu().numpy(), O.mx_pack(q))


@pytest.mark.parametrize("st", ["f32", "bf16"])
def test_norm_to_mxfp4_next_to_the_borders(st):
    """Weights that put every n within a float32 step of a code's border, on either side."""
    rng = np.random.default_rng(11)
    H = 2048
    y = torch.as_tensor(rng.standard_normal((1, H)) + np.sign(rng.standard_normal((1, H)))).to(TORCH[st])
    s = _f(y)
    pre = 1 / np.sqrt((s * s).mean() + 1e-6)
    border = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], (1, H))
    border[0, ::32] = 5.0  # the block's largest lies in [4, 8): scale 1
    w = torch.as_tensor((border / (s * pre))[0]).float()
    n = L.mx_empty(1, H)
    L.block_norm(y.cuda(), n=n, pre_w=w.cuda())
    _, nv = O.block_norm64(s, pre_w=w.double().numpy())
    assert 0.3 < (np.abs(nv) < border).mean() < 0.7
    q, sc = O.mx_quantize64(nv)
    assert np.array_equal(n.scales.cpu().numpy(), sc) and np.array_equal(n.codes.cpu().numpy(), O.mx_pack(q))


def test_rows_alone_zeros_and_values_that_are_not_finite():
    x = torch.randn((4, 64), device="cuda")
    x[1] = 0
    x[2, 9] = float("nan")
    x[3, 40] = float("inf")
    w = torch.ones(64, device="cuda")
    n, q = torch.empty_like(x), L.mx_empty(4, 64)
    L.block_norm(x, n=n, pre_w=w)
    L.block_norm(x, n=q, pre_w=w)
    assert n[0].isfinite().all() and n[1].eq(0).all() and n[2].isnan().all()
    assert n[3, 40].isnan() and n[3, :40].eq(0).all() and n[3, 41:].eq(0).all()  # inf / inf, finite / inf
    assert q.scales.cpu().tolist()[1:] == [[0, 0], [255, 255], [0, 255]]
    assert q.codes[1:].eq(0).all() or (q.codes[1:] & 0x77).eq(0).all()  # zeros, of either sign


def test_captured_and_replayed():
    y, r, w = (torch.randn(s, device="cuda") for s in ((6, 224), (6, 224), (224,)))
    r_out, n = torch.empty_like(r), L.mx_empty(6, 224)
    L.block_norm(y, r, r_out, n, pre_w=w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.block_norm(y, r, r_out, n, pre_w=w)
    for _ in range(3):
        y.normal_()
        want, wr = L.mx_empty(6, 224), torch.empty_like(r)
        L.block_norm(y, r, wr, want, pre_w=w)
        n.codes.zero_(), r_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n.codes, want.codes) and torch.equal(n.scales, want.scales) and torch.equal(r_out, wr)
