"""block_norm on the GPU: calls that lie beside those of test_gpu_norm.py."""
import itertools

import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
from mx_bounds import HALF_STEP, TORCH, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nt", ["same", "mx"])
@pytest.mark.parametrize("M,H,t", [(3, 96, "f32"), (5, 7168, "bf16"), (300, 7168, "f32"), (600, 7168, "bf16"),
                                   (2, 32768, "f32"), (530, 16384, "bf16")])
def test_the_residual_stream_normed_onto_itself(M, H, t, nt):
    """y, r and r_out one tensor: the bits of the call on three."""
    rng = np.random.default_rng(M + H)
    x = torch.as_tensor(rng.standard_normal((M, H))).to(TORCH[t]).cuda()
    w = torch.as_tensor(rng.standard_normal(H)).to(TORCH[t]).cuda()
    kw = dict(pre_w=w, post_w=w, gate=w.clone(), alpha=0.5)
    out = lambda: L.mx_empty(M, H) if nt == "mx" else torch.empty_like(x)  # noqa: E731
    s, n, z, m = torch.empty_like(x), out(), x.clone(), out()
    L.block_norm(x, x.clone(), s, n, **kw)
    L.block_norm(z, z, z, m, **kw)
    assert torch.equal(z, s)
    if nt == "mx":
        assert torch.equal(m.codes, n.codes) and torch.equal(m.scales, n.scales)
    else:
        assert torch.equal(m, n)


def _codes_are_float64s(n, nv):
    q, sc = O.mx_quantize64(nv)
    wrong = int((n.scales.cpu().numpy() != sc).sum()), int((n.codes.cpu().numpy() != O.mx_pack(q)).sum())
    assert wrong == (0, 0), f"{wrong} scales and pairs of codes of {sc.size} and {q.size // 2}"


def _f(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("eps", [0.0, 1e-40])
@pytest.mark.parametrize("se,we", [(-75, -68), (-60, -80), (-100, 60), (60, -100), (100, -60), (-20, -20), (-40, -90)])
@pytest.mark.parametrize("M,H,t", [(3, 4096, "f32"), (600, 2304, "bf16")])
def test_codes_of_very_small_and_large_rows(M, H, t, se, we, eps):
    """s and pre_w whose product leaves float32's normal range where s / rms(s) * pre_w does not."""
    rng = np.random.default_rng(abs(se - 3 * we + M))
    y = torch.as_tensor(np.ldexp(rng.standard_normal((M, H)), se)).to(TORCH[t])
    w = torch.as_tensor(np.ldexp(rng.standard_normal(H), we)).to(TORCH[t])
    n = L.mx_empty(M, H)
    L.block_norm(y.cuda(), n=n, pre_w=w.cuda(), eps=eps)
    _codes_are_float64s(n, O.block_norm64(_f(y), eps=eps, pre_w=_f(w))[1])


@pytest.mark.parametrize("ye,pe,ge", [(100, 40, -30), (-100, -40, 30), (-60, -30, -40), (-100, -40, 90), (60, 60, 60)])
@pytest.mark.parametrize("M,H", [(3, 4096), (600, 2304)])
def test_products_of_bf16_values_outside_float32s_range(M, H, ye, pe, ge):
    """y * post_w * gate leaves float32's range where y / rms(y) * post_w * gate does not."""
    rng = np.random.default_rng(abs(ye + 3 * pe) + M)
    t = lambda e, *s: torch.as_tensor(np.ldexp(rng.standard_normal(s), e)).bfloat16()  # noqa: E731
    y, post, gate, pre = t(ye, M, H), t(pe, H), t(ge, M, H), t(0, H)
    s, n = torch.empty((M, H), dtype=torch.bfloat16, device="cuda"), L.mx_empty(M, H)
    L.block_norm(y.cuda(), r_out=s, n=n, pre_w=pre.cuda(), post_w=post.cuda(), gate=gate.cuda(), eps=0.0)
    stored = lambda v: torch.as_tensor(v).float().bfloat16().double().numpy()  # noqa: E731
    sv, nv = O.block_norm64(_f(y), None, _f(post), _f(gate), 1.0, 0.0, _f(pre), stored)
    assert np.isfinite(stored(sv)).all() and np.array_equal(_f(s), stored(sv))
    _codes_are_float64s(n, nv)


@pytest.mark.parametrize("yt,rt,wt", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("bf16", "f32", "bf16"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("M,H", [(3, 96), (300, 2304), (5, 8224)])
def test_every_combination_of_the_optional_tensors(M, H, yt, rt, wt):
    """r, post_w, gate, r_out and n, each there or not; n as values and as MXFP4."""
    rng = np.random.default_rng(M + H)
    t = lambda ty, *s: torch.as_tensor(rng.standard_normal(s)).to(TORCH[ty]).cuda()  # noqa: E731
    y, res, pre, post, gates = t(yt, M, H), t(rt, M, H), t(wt, H), t(wt, H), {"channel": t(wt, H), "row": t(wt, M, H)}
    for has_r, has_post, gate, out in itertools.product((0, 1), (0, 1), (None, "channel", "row"), ("r", "n", "rn", "mx", "rmx")):
        r, pw, g = res if has_r else None, post if has_post else None, gates.get(gate)
        st = rt if has_r or "r" in out else yt  # s's type
        r_out = torch.full((M, H), float("nan"), dtype=TORCH[st], device="cuda") if "r" in out else None
        n = L.mx_empty(M, H) if "mx" in out else torch.empty((M, H), device="cuda") if "n" in out else None
        L.block_norm(y, r, r_out, n, pre_w=None if n is None else pre, post_w=pw, gate=g, alpha=0.75)
        stored = lambda v: torch.as_tensor(v).float().to(TORCH[st]).double().numpy()  # noqa: E731
        f = lambda v: None if v is None else _f(v)  # noqa: E731
        s, nv = O.block_norm64(_f(y), f(r), f(pw), f(g), 0.75, 1e-6, _f(pre), stored)
        what = f"r {has_r} post {has_post} gate {gate} out {out}"
        if "mx" in out:
            _codes_are_float64s(n, nv)
            assert r_out is None or np.array_equal(_f(r_out), stored(s)), what
            continue
        part = np.abs(s - (f(r) if has_r else 0.0))
        b = 2.0 ** -18 * part + 2.0 ** -23 * np.abs(s)
        step = HALF_STEP[TORCH[st]]
        if r_out is not None:
            check(r_out, s, b + step * (np.abs(s) + b) + 1e-37, what)
        if n is not None:
            # s may be stored a step off what float64 stores (b and the type's rounding), which moves its mean and itself
            ds = b + step * (np.abs(s) + b)
            rms = np.sqrt((stored(s) ** 2).mean(1, keepdims=True) + 1e-6)
            moved = np.sqrt((ds ** 2).mean(1, keepdims=True)) / rms
            lim = 2 * ((ds + np.abs(s) * moved) / rms * np.abs(_f(pre))) + (2.0 ** -18 + 2.0 ** -24) * np.abs(nv)
            check(n, nv, lim / (1 - moved) + 1e-37, what)
