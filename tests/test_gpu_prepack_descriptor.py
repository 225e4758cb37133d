"""w4a16_prepack with one descriptor for the source and the result."""
import ctypes

import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
from helpers import grouped_words

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,K,N", [(1, 64, 64), (3, 256, 320)])
def test_prepack_into_the_source_descriptor(E, K, N):
    """`out` may be `src`: the kernel reads the codes that the descriptor named before the call."""
    q = np.random.default_rng(K).integers(-2 ** 31, 2 ** 31, (E, K // 8, N)).astype(np.int32)
    qw, scales = torch.as_tensor(q).cuda(), torch.ones((E, K // 32, N), device="cuda")
    dst = torch.full_like(qw, 0x55555555)
    d = L.WeightDesc(qw.data_ptr(), scales.data_ptr(), K, N, 32, E, L.LAYOUT_CANONICAL)
    st = L.load_library().w4a16_prepack(ctypes.byref(d), dst.data_ptr(), dst.numel() * 4, ctypes.byref(d),
                                        torch.cuda.current_stream().cuda_stream)
    assert st == L.OK
    assert (d.qw, d.scales, d.K, d.N, d.layout) == (dst.data_ptr(), scales.data_ptr(), K, N, L.LAYOUT_GROUPED)
    assert np.array_equal(dst.cpu().numpy().ravel(), grouped_words(q).ravel())
