"""CPU checks of the MXFP4 and norm entry points: the oracle against the format's own
definition, refusals of the C ABI (nothing is enqueued: these pointers are not device memory)
and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


# ---------------------------------------------------------------- the oracle

def test_codes_are_the_nearest_values_ties_to_even():
    x = np.zeros((1, 32))
    pairs = {0.0: 0, 0.2: 0, 0.25: 0, 0.26: 1, 0.5: 1, 0.75: 2, 1.25: 2, 1.26: 3, 1.75: 4, 2.5: 4, 2.51: 5, 3.5: 6, 5.0: 6,
             5.01: 7, 6.0: 7, 7.9: 7, 4.0: 6}
    for i, v in enumerate(pairs):
        x[0, i] = -v if i % 2 else v
    q, s = O.mx_quantize64(x)
    assert s.tolist() == [[127]]  # 7.9 lies in [4, 8): scale 1
    for i, c in enumerate(pairs.values()):
        assert q[0, i] == c + 8 * (i % 2), list(pairs)[i]


@pytest.mark.parametrize("amax,byte", [(0.0, 0), (2.0 ** -130, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (1.0, 125),
                                       (3.999, 126), (4.0, 127), (2.0 ** 127, 252)])
def test_scale_bytes(amax, byte):
    x = np.full((1, 32), amax)
    assert O.mx_quantize64(x)[1].tolist() == [[byte]]


def test_values_come_back_and_a_nan_byte_is_its_block_alone():
    rng = np.random.default_rng(0)
    q = rng.integers(0, 16, (3, 64)).astype(np.uint8)
    s = rng.integers(1, 254, (3, 2)).astype(np.uint8)
    v = O.mx_values64(O.mx_pack(q), s)
    mag = {0: 0, 1: 0.5, 2: 1, 3: 1.5, 4: 2, 5: 3, 6: 4, 7: 6}
    for r, k in ((0, 0), (1, 33), (2, 63)):
        assert v[r, k] == (-1) ** (int(q[r, k]) >> 3) * mag[int(q[r, k]) & 7] * 2.0 ** (int(s[r, k // 32]) - 127)
    s[1, 0] = 255
    assert np.isnan(O.mx_values64(O.mx_pack(q), s)).nonzero()[0].tolist() == [1] * 32


# ---------------------------------------------------------------- the C ABI

def _mx(rows=64, K=256, layout=L.MX_TILED, codes=0x100000, scales=0x200000):
    return L.MxDesc(codes, scales, rows, K, layout)


def _p(v):
    return ctypes.c_void_p(v)


def test_sizes(lib):
    assert lib.w4a16_mx_codes_bytes(5, 96, L.MX_ROWS) == 5 * 48 and lib.w4a16_mx_scales_bytes(5, 96, L.MX_ROWS) == 15
    assert lib.w4a16_mx_codes_bytes(80, 160, L.MX_TILED) == 2 * 2 * 4096
    assert lib.w4a16_mx_scales_bytes(80, 160, L.MX_TILED) == 2 * 2 * 256
    for rows, K, layout in ((5, 40, 0), (-1, 32, 0), (5, 32, 1), (16, 32, 2), (16, (1 << 20) + 32, 0), ((1 << 24) + 1, 32, 0)):
        assert lib.w4a16_mx_codes_bytes(rows, K, layout) == 0 == lib.w4a16_mx_scales_bytes(rows, K, layout)


def test_quantize_refusals(lib):
    def call(x=0x1000, xt=0, rows=4, K=64, c=0x100000, cb=128, s=0x200000, sb=8, fn=lib.w4a16_mx_quantize):
        return fn(_p(x), xt, rows, K, _p(c), cb, _p(s), sb, None)
    assert call(rows=0, x=0) == L.OK
    for kw in (dict(x=0), dict(x=0x1008), dict(xt=2), dict(rows=-1), dict(c=0), dict(s=0),
               dict(s=0x200004)):
        assert call(**kw) == L.ERR_INVALID_ARG, kw
    assert call(cb=127) == call(sb=7) == L.ERR_WORKSPACE
    for kw in (dict(K=48), dict(K=(1 << 20) + 32)):
        assert call(**kw) == L.ERR_UNSUPPORTED, kw
    qw = lambda **kw: lib.w4a16_mx_quantize_weight(_p(kw.get("w", 0x1000)), kw.get("wt", 0), kw.get("K", 64), 4,  # noqa: E731
                                                   _p(0x100000), kw.get("cb", 128), _p(0x200000), 8, None)
    assert qw(w=0) == qw(wt=5) == qw(K=-32) == L.ERR_INVALID_ARG and qw(K=33) == L.ERR_UNSUPPORTED
    assert qw(cb=100) == L.ERR_WORKSPACE


def test_prepack_and_dequantize_refusals(lib):
    src, out = _mx(64, 256, L.MX_ROWS), L.MxDesc()
    call = lambda s=src, c=0x300000, cb=8192, sc=0x400000, sb=512, o=out: lib.w4a16_mx_prepack(  # noqa: E731
        ctypes.byref(s), _p(c), cb, _p(sc), sb, ctypes.byref(o) if o is not None else None, None)
    for kw in (dict(c=0), dict(o=None), dict(c=0x100800), dict(sc=0x300010),
               dict(s=_mx(64, 256, L.MX_ROWS, codes=0)), dict(s=_mx(64, 256, L.MX_ROWS, scales=0x200004))):
        assert call(**kw) == L.ERR_INVALID_ARG, kw
    assert call(cb=8191) == call(sb=511) == L.ERR_WORKSPACE
    assert call(s=_mx()) == call(s=_mx(63, 256, L.MX_ROWS)) == call(s=_mx(64, 40, L.MX_ROWS)) == L.ERR_UNSUPPORTED
    deq = lambda m, o=0x300000, t=0, n=1 << 30: lib.w4a16_mx_dequantize(ctypes.byref(m), _p(o), t, n, None)  # noqa: E731
    assert deq(src, o=0) == deq(src, t=2) == L.ERR_INVALID_ARG and deq(src, n=64 * 256 * 4 - 1) == L.ERR_WORKSPACE
    assert deq(_mx(layout=7)) == L.ERR_UNSUPPORTED
    assert lib.w4a16_mx_dequantize(None, _p(0x1000), 0, 64, None) == L.ERR_INVALID_ARG


@pytest.mark.parametrize("a4", [False, True])
def test_gemm_refusals(lib, a4):
    w = _mx(64, 256)
    ws = (lib.w4a16_mx_gemm_a4_workspace_bytes(4, ctypes.byref(w)) if a4
          else lib.w4a16_mx_gemm_workspace_bytes(4, L.BF16, ctypes.byref(w)))
    assert ws > 0

    def call(M=4, xt=L.BF16, w=w, x=0x300000, y=0x400000, yt=L.F32, wsp=0x500000, n=ws, xK=256, xl=L.MX_ROWS, xs=0x600000):
        if a4:
            xd = _mx(M, xK, xl, x, xs)
            return lib.w4a16_mx_gemm_a4(ctypes.byref(xd), ctypes.byref(w), _p(y), yt, _p(wsp), n, None)
        return lib.w4a16_mx_gemm(_p(x), xt, M, ctypes.byref(w), _p(y), yt, _p(wsp), n, None)
    assert call(M=0, x=0) == L.OK
    for kw in (dict(M=-1), dict(x=0), dict(x=0x300008), dict(y=0), dict(y=0x400004), dict(yt=3), dict(wsp=0),
               dict(y=0x300010), dict(w=_mx(codes=0)), dict(w=_mx(scales=0x200008))) + (
                   (dict(xs=0), dict(y=0x600000)) if a4 else (dict(xt=2),)):
        assert call(**kw) == L.ERR_INVALID_ARG, kw
    for kw in (dict(w=_mx(layout=L.MX_ROWS)), dict(w=_mx(rows=72)), dict(w=_mx(K=72)), dict(w=_mx(layout=3))) + (
            (dict(xK=128), dict(xl=L.MX_TILED, M=16)) if a4 else ()):
        assert call(**kw) == L.ERR_UNSUPPORTED, kw
    assert call(n=ws - 1) == L.ERR_WORKSPACE


@pytest.mark.parametrize("a4", [False, True])
def test_mlp_refusals(lib, a4):
    g, u, d = _mx(512, 256), _mx(512, 256), _mx(256, 512)
    r = ctypes.byref
    size = (lambda g, u, d, M=4: lib.w4a16_mx_swiglu_mlp_a4_workspace_bytes(M, r(g), r(u), r(d))) if a4 else (
        lambda g, u, d, M=4: lib.w4a16_mx_swiglu_mlp_workspace_bytes(M, L.F32, r(g), r(u), r(d)))
    ws = size(g, u, d)
    assert ws > 0 and size(g, u, g) == 0 and size(g, u, d, 0) == 0 and size(g, d, d) == 0

    def call(g=g, u=u, d=d, x=0x300000, y=0x400000, n=ws):
        if a4:
            return lib.w4a16_mx_swiglu_mlp_a4(r(_mx(4, 256, L.MX_ROWS, x)), r(g), r(u), r(d), _p(y), 0, _p(0x500000), n, None)
        return lib.w4a16_mx_swiglu_mlp(_p(x), L.F32, 4, r(g), r(u), r(d), _p(y), 0, _p(0x500000), n, None)
    assert call(d=_mx(256, 256)) == call(u=_mx(512, 288)) == call(g=_mx(512, 256, L.MX_ROWS)) == L.ERR_UNSUPPORTED
    assert call(x=0) == call(y=0) == call(y=0x300000) == call(d=_mx(256, 512, codes=0)) == L.ERR_INVALID_ARG
    assert call(n=ws - 1) == L.ERR_WORKSPACE


def _norm(**kw):
    a = dict(y=0x100000, r=0x200000, r_out=0x300000, post_w=None, pre_w=0x400000, gate=None, gate_rows=1, n=0x500000,
             n_codes=None, n_scales=None, y_type=0, r_type=0, w_type=0, n_type=0, alpha=1.0, eps=1e-6)
    a.update(kw)
    return L.NormDesc(**a)


def test_norm_refusals(lib):
    call = lambda M=4, H=64, **kw: lib.w4a16_block_norm(ctypes.byref(_norm(**kw)), M, H, None)  # noqa: E731
    assert call(M=0) == call(H=0) == L.OK
    mx = dict(n=None, n_codes=0x500000, n_scales=0x600000)
    for kw in (dict(y=None), dict(pre_w=None), dict(n=None, r_out=None), dict(n_codes=0x600000), dict(mx, n_scales=None),
               dict(mx, n=0x700000), dict(y_type=2), dict(r_type=-1), dict(w_type=9), dict(n_type=4), dict(y=0x100004),
               dict(n=0x500008), dict(gate=0x600000, gate_rows=3), dict(n=0x100010), dict(r_out=0x200010),
               dict(n=0x300000), dict(gate=0x500100), dict(post_w=0x300010), dict(M=-1), dict(H=-8)):
        assert call(**kw) == L.ERR_INVALID_ARG, kw
    for kw in (dict(H=60), dict(H=40, **mx), dict(H=32768 + 8), dict(M=(1 << 24) + 1)):
        assert call(**kw) == L.ERR_UNSUPPORTED, kw
    assert lib.w4a16_block_norm(None, 4, 64, None) == L.ERR_INVALID_ARG


# ---------------------------------------------------------------- the binding

def _m(rows, K, layout=L.MX_ROWS):
    lib = L.load_library()
    return L.MxMatrix(torch.zeros(lib.w4a16_mx_codes_bytes(rows, K, layout), dtype=torch.uint8),
                      torch.zeros(lib.w4a16_mx_scales_bytes(rows, K, layout), dtype=torch.uint8), rows, K, layout)


def test_binding_refuses_wrong_tensors():
    w, ws = _m(64, 128, L.MX_TILED), torch.zeros(256, dtype=torch.uint8)
    short = L.MxMatrix(w.codes[:-1], w.scales, 64, 128, L.MX_TILED)
    for m in (short, L.MxMatrix(w.codes, w.scales, 64, 256, L.MX_TILED), L.MxMatrix(w.codes, w.scales, 64, 130)):
        with pytest.raises(ValueError):
            L.mx_gemm(torch.zeros((2, 128)), m, torch.zeros((2, 64)), ws)
    with pytest.raises(TypeError):
        L.mx_gemm(torch.zeros((2, 128)), L.MxMatrix(w.codes.int(), w.scales, 64, 128, 1), torch.zeros((2, 64)), ws)
    with pytest.raises(ValueError):  # host memory
        L.mx_gemm(torch.zeros((2, 128)), w, torch.zeros((2, 64)), ws)
    with pytest.raises(ValueError):
        L.mx_quantize(torch.zeros((2, 128)), _m(2, 128))
    with pytest.raises(TypeError):
        L.mx_quantize(torch.zeros((2, 128), dtype=torch.float16), _m(2, 128))
    with pytest.raises(ValueError):
        L.mx_empty(5, 40, device="cpu")


class _OnDevice(torch.Tensor):
    """A host tensor that says it is on device 0 (1: `_OnAnother`)."""
    index = 0

    def get_device(self):
        return self.index


class _OnAnother(_OnDevice):
    index = 1


def _dev(t, cls=_OnDevice):
    return t.as_subclass(cls)


@pytest.fixture
def no_calls(monkeypatch):
    """The current device is 0, and no entry point may be reached."""
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    monkeypatch.setattr(L, "_stream_of", lambda *a: pytest.fail("the library was reached"))
    monkeypatch.setattr(L, "_stream", lambda s: pytest.fail("the library was reached"))


def _dm(rows, K, layout=L.MX_ROWS):
    m = _m(rows, K, layout)
    return L.MxMatrix(_dev(m.codes), _dev(m.scales), rows, K, layout)


def test_binding_refuses_other_shapes_and_devices(no_calls):
    w, ws, z = _dm(64, 128, L.MX_TILED), _dev(torch.zeros(256, dtype=torch.uint8)), lambda *s: _dev(torch.zeros(s))
    for x, y in ((z(2, 96), z(2, 64)), (z(2, 128), z(3, 64)), (z(2, 128), z(2, 60)), (_dm(2, 128), z(3, 64)),
                 (z(128, 2).t(), z(2, 64)), (_dev(torch.zeros(2, 128), _OnAnother), z(2, 64)),
                 (z(2, 128), _dev(torch.zeros(2, 64), _OnAnother))):
        with pytest.raises(ValueError):
            L.mx_gemm(x, w, y, ws)
    elsewhere = L.MxMatrix(w.codes, _dev(w.scales.as_subclass(torch.Tensor), _OnAnother), 64, 128, L.MX_TILED)
    with pytest.raises(ValueError):
        L.mx_gemm(z(2, 128), elsewhere, z(2, 64), ws)
    with pytest.raises(ValueError):
        L.mx_swiglu_mlp(z(2, 128), w, elsewhere, _dm(128, 64, L.MX_TILED), z(2, 128), ws)
    with pytest.raises(ValueError):
        L.mx_quantize(z(2, 128), _dm(2, 96))
    with pytest.raises(ValueError):
        L.mx_prepack(_dm(64, 128), _dm(64, 160, L.MX_TILED))
    with pytest.raises(ValueError):
        L.mx_dequantize(_dm(64, 128), z(64, 96))


def test_binding_refuses_norm_arguments(no_calls):
    z = lambda *s, t=torch.float32: _dev(torch.zeros(s, dtype=t))  # noqa: E731
    y, w = z(3, 64), z(64)
    for kw in (dict(r=z(2, 64)), dict(r_out=z(3, 32)), dict(n=z(3, 96)), dict(n=_dm(4, 64)), dict(pre_w=z(32)),
               dict(gate=z(2, 64)), dict(post_w=z(1, 64)), dict(n=_dev(torch.zeros(3, 64), _OnAnother))):
        with pytest.raises(ValueError):
            L.block_norm(y, **{"n": z(3, 64), "pre_w": w, **kw})
    for kw in (dict(r=z(3, 64), r_out=z(3, 64, t=torch.bfloat16)), dict(post_w=z(64, t=torch.bfloat16)),
               dict(n=z(3, 64, t=torch.float16))):
        with pytest.raises(TypeError):
            L.block_norm(y, **{"n": z(3, 64), "pre_w": w, **kw})


def test_overlaps_are_refused(lib):
    """Outputs and workspaces that overlap an input, a weight or each other."""
    q = lambda x, c, s: lib.w4a16_mx_quantize(_p(x), 0, 4, 64, _p(c), 128, _p(s), 8, None)  # noqa: E731
    assert q(0x1000, 0x1010, 0x2000) == q(0x1000, 0x2000, 0x13f0) == q(0x1000, 0x2000, 0x2070) == L.ERR_INVALID_ARG
    qw = lambda w, c, s: lib.w4a16_mx_quantize_weight(_p(w), 1, 64, 4, _p(c), 128, _p(s), 8, None)  # noqa: E731
    assert qw(0x1000, 0x11f0, 0x2000) == qw(0x1000, 0x2000, 0x1000) == L.ERR_INVALID_ARG
    for layout in (L.MX_ROWS, L.MX_TILED):
        m = _mx(64, 256, layout, 0x100000, 0x200000)
        for out in (0x100000, 0x101ff0, 0x200000, 0x200000 - 64 * 256 * 2 + 16):
            assert lib.w4a16_mx_dequantize(ctypes.byref(m), _p(out), L.BF16, 1 << 20, None) == L.ERR_INVALID_ARG
    w, r = _mx(64, 256, codes=0x100000, scales=0x200000), ctypes.byref
    g, d = _mx(256, 256, codes=0x700000, scales=0x800000), _mx(256, 256, codes=0x900000, scales=0xa00000)
    n = lib.w4a16_mx_gemm_workspace_bytes(40, L.F32, r(w))
    for y, ws in ((0x101ff0, 0x500000), (0x2001f0, 0x500000), (0x400000, 0x300000), (0x400000, 0x400000),
                  (0x400000, 0x100000), (0x400000, 0x200000)):
        assert lib.w4a16_mx_gemm(_p(0x300000), L.F32, 40, r(w), _p(y), 0, _p(ws), n, None) == L.ERR_INVALID_ARG, (y, ws)
    n = lib.w4a16_mx_swiglu_mlp_workspace_bytes(4, L.BF16, r(g), r(g), r(d))
    for y, ws in ((0x900000, 0x500000), (0xa00000, 0x500000), (0x400000, 0x700010), (0x400000, 0x400010)):
        assert lib.w4a16_mx_swiglu_mlp(_p(0x300000), L.BF16, 4, r(g), r(g), r(d), _p(y), 0, _p(ws), n,
                                       None) == L.ERR_INVALID_ARG, (y, ws)


def test_empty_matrices_need_no_pointers(lib):
    r, out = ctypes.byref, L.MxDesc()
    for rows, K in ((0, 64), (16, 0), (0, 0)):
        m = _mx(rows, K, L.MX_ROWS, 0, 0)
        assert lib.w4a16_mx_dequantize(r(m), None, 0, 0, None) == L.OK
        assert lib.w4a16_mx_prepack(r(m), None, 0, None, 0, r(out), None) == L.OK
        assert (out.rows, out.K, out.layout) == (rows, K, L.MX_TILED)
        if rows == 0:
            assert lib.w4a16_mx_gemm(None, 0, 4, r(out), None, 0, None, 0, None) == L.OK
    w = _mx(16, 0, codes=0, scales=0)  # an empty sum still has its y
    assert lib.w4a16_mx_gemm(None, 0, 4, r(w), None, 0, None, 0, None) == L.ERR_INVALID_ARG
    assert lib.w4a16_mx_gemm(None, 0, 4, r(w), _p(0x1008), 0, None, 0, None) == L.ERR_INVALID_ARG
