"""CPU checks of refusals of the MXFP4 calls and block_norm: tensors that lie on one another, and sizes
past the limits (nothing is enqueued: these pointers are not device memory)."""
import ctypes

import pytest
import torch

import int4_w4a16_group_g32_amd as L


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


R = 0x200000  # r and r_out


def _norm(lib, M=4, H=64, **kw):
    a = dict(y=0x100000, r=R, r_out=R, post_w=None, pre_w=0x400000, gate=None, gate_rows=1, n=0x500000, n_codes=None,
             n_scales=None, y_type=L.F32, r_type=L.F32, w_type=L.F32, n_type=L.F32, alpha=1.0, eps=1e-6)
    a.update(kw)
    return lib.w4a16_block_norm(ctypes.byref(L.NormDesc(**a)), M, H, None)


@pytest.mark.parametrize("kw", [
    dict(gate=R), dict(gate=R, gate_rows=4), dict(gate=R, w_type=L.BF16), dict(gate=R + 256), dict(post_w=R), dict(pre_w=R),
    dict(pre_w=R + 512), dict(y=R, r_type=L.BF16), dict(y=R, y_type=L.BF16), dict(y=R + 16), dict(y=R, r=None),
    dict(n=R), dict(y=R, n=R), dict(n=None, n_codes=R, n_scales=0x600000), dict(n=None, n_codes=0x500000, n_scales=R)])
def test_an_input_in_place_of_the_residual_is_refused(lib, kw):
    """Only r itself (and y of its type) may be where r_out is: whatever other rows read too may not."""
    assert _norm(lib, **kw) == L.ERR_INVALID_ARG


@pytest.mark.parametrize("M,rows,K", [(1 << 14, 1 << 20, 8192), (513, 1 << 24, 32), (1 << 24, 528, 32),
                                      (1 << 24, 1 << 24, 32)])
def test_products_of_more_values_than_the_limit_have_no_workspace_size(lib, M, rows, K):
    """M * N above 2^33: the call is refused, and its size is 0."""
    w = L.MxDesc(0x100000, 0x200000, rows, K, L.MX_TILED)
    p, r = ctypes.c_void_p, ctypes.byref
    x = L.MxDesc(0x300000, 0x400000, M, K, L.MX_ROWS)
    for xt in (L.F32, L.BF16):
        assert lib.w4a16_mx_gemm_workspace_bytes(M, xt, r(w)) == 0
        assert lib.w4a16_mx_gemm(p(0x300000), xt, M, r(w), p(0x500000), L.F32, p(0x600000), 1 << 40, None) == L.ERR_UNSUPPORTED
    assert lib.w4a16_mx_gemm_a4_workspace_bytes(M, r(w)) == 0
    assert lib.w4a16_mx_gemm_a4(r(x), r(w), p(0x500000), L.F32, p(0x600000), 1 << 40, None) == L.ERR_UNSUPPORTED


class _OnDevice(torch.Tensor):
    """A host tensor that says it is on device 0."""

    def get_device(self):
        return 0


def test_what_is_no_tensor_is_a_type_error(lib, monkeypatch):
    """Outputs, workspaces and a matrix's parts, as in the other calls."""
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    monkeypatch.setattr(L, "_stream_of", lambda *a: pytest.fail("the library was reached"))
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t).as_subclass(_OnDevice)  # noqa: E731
    w = L.MxMatrix(z(8192, t=torch.uint8), z(512, t=torch.uint8), 128, 128, L.MX_TILED)
    x, y, ws = z(2, 128), z(2, 128), z(256, t=torch.uint8)
    for bad in (L.MxMatrix(None, w.scales, 128, 128, L.MX_TILED), L.MxMatrix(w.codes, None, 128, 128, L.MX_TILED)):
        with pytest.raises(TypeError):
            L.mx_gemm(x, bad, y, ws)
    for a, b in ((None, ws), (y, None)):
        with pytest.raises(TypeError):
            L.mx_gemm(x, w, a, b)
        with pytest.raises(TypeError):
            L.mx_swiglu_mlp(x, w, w, w, a, b)
