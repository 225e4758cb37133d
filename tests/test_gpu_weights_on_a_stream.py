"""quantize_to_weight on another stream than the current one."""
import pytest
import torch

import int4_w4a16_group_g32_amd as L

pytestmark = pytest.mark.gpu


def test_weights_quantized_on_another_stream():
    """Their canonical codes are freed while that stream still works: the current stream's tensors are not put there."""
    torch.manual_seed(2)
    w = torch.randn((4096, 4096), device="cuda")
    want = L.quantize_to_weight(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [L.quantize_to_weight(w, side) for _ in range(3)]
    other = [torch.full((512, 4096), 255, dtype=torch.int32, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(g.qw, want.qw) and torch.equal(g.scales, want.scales) for g in got)
    assert all(o.eq(255).all() for o in other)


def test_weights_made_on_another_stream_and_freed_while_in_use():
    """The next weights made there are not put over them before the current stream's product, still
    waiting behind other work, has read them."""
    torch.manual_seed(5)
    a, b = torch.randn((4096, 4096), device="cuda"), torch.randn((4096, 4096), device="cuda")
    x, busy = torch.randn((4, 4096), device="cuda"), torch.randn((4096, 4096), device="cuda")
    first = L.quantize_to_weight(a)
    ws = L.new_workspace(L.gemm_workspace_bytes(4, first, L.F32))
    want, y = torch.empty((4, 4096), device="cuda"), torch.empty((4, 4096), device="cuda")
    L.gemm(x, first, want, ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    w = L.quantize_to_weight(a, side)
    torch.cuda.synchronize()
    for _ in range(40):
        torch.mm(busy, busy, out=b)  # some 40 ms
    L.gemm(x, w, y, ws)
    del w
    other = [L.quantize_to_weight(busy, side) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and len(other) == 3
