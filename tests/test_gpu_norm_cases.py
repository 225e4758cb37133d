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
