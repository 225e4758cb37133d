"""block_norm on the GPU: calls that lie beside those of test_gpu_norm.py."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O
from mx_bounds import TORCH

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
