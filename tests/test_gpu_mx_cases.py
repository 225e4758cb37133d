"""MXFP4 on the GPU: calls that lie beside those of test_gpu_mx.py."""
import ctypes

import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O

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
