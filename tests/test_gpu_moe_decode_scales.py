"""An expert whose scales are not finite reaches the tokens that chose it and no others,
as in w4a16_moe_grouped: in the long product over the chosen experts, the rows of the other
tokens are zeros there, and zero times infinity must not count."""
import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import workloads as W
from test_gpu_lora import _code, _x
from test_gpu_moe_decode import _device, _run, _stacks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", [0, 1, 2])  # gate, up, down
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("M,H,I,E,k,shared", [(2, 128, 64, 4, 1, False), (4, 128, 192, 6, 2, True),
                                              (8, 256, 704, 12, 3, False), (16, 512, 320, 20, 4, True),
                                              (16, 64, 2048, 9, 2, False), (6, 2560, 64, 300, 32, True)])
def test_scales_that_are_not_finite(M, H, I, E, k, shared, which, value, dtype):
    M = min(M, 8 if dtype == "f32" else 16)
    stacks = _stacks(E, H, I, 700)
    sh = _device(_stacks(1, H, I, 701)) if shared else None
    x, lg = _x(M, H, dtype, 702), W.router_logits(M, E, 703).cuda()
    want, ids, w = _run(x, lg, k, _device(stacks), torch.float32, sh)
    assert bool((w > 0).all())
    bad = int(ids[0, 0])
    hit = (ids == bad).any(1)
    assert bool(torch.isfinite(want).all())
    q, s = stacks[which]
    s = s.copy()
    s[bad] = value
    stacks[which] = (q, s)
    got = _run(x, lg, k, _device(stacks), torch.float32, sh, out=False)
    assert torch.equal(got[~hit], want[~hit])
    assert not bool(torch.isfinite(got[hit]).any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_group_of_the_down_projection(dtype):
    """Infinite scales in one group of one expert: its tokens' columns, as w4a16_moe_grouped gives them."""
    M, H, I, E, k = 8, 128, 256, 8, 2
    stacks = _stacks(E, H, I, 710)
    x, lg = _x(M, H, dtype, 711), W.router_logits(M, E, 712).cuda()
    want, ids, w = _run(x, lg, k, _device(stacks), torch.float32)
    bad = int(ids[3, 1])
    q, s = stacks[2]
    s = s.copy()
    s[bad, 5, 64:] = np.inf
    ws3 = _device([stacks[0], stacks[1], (q, s)])
    got = _run(x, lg, k, ws3, torch.float32, out=False)
    y = torch.empty((M, H), device="cuda")
    L.moe_grouped(x, ids, w, *ws3, y, L.new_workspace(L.moe_workspace_bytes(M, k, _code(dtype), *ws3)))
    torch.cuda.synchronize()
    hit = (ids == bad).any(1)
    assert torch.equal(got[~hit], want[~hit]) and torch.equal(got[:, :64], want[:, :64])
    assert not bool(torch.isfinite(got[hit][:, 64:]).any())
    assert torch.equal(torch.isfinite(got), torch.isfinite(y))
