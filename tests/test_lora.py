"""CPU checks of the low-rank-adapter entry points: the oracle against loops and
closed forms, and every refusal (nothing is enqueued: the pointers are not device
memory)."""
import ctypes

import numpy as np
import pytest
import torch

import int4_w4a16_group_g32_amd as L
import oracle as O


def _codes(K, N, seed):
    return O.quantize_w4a16((np.random.default_rng(seed).standard_normal((K, N)) * 0.02).astype(np.float32))


def _lora(n, R, K, N, seed, ranks=None):
    r = np.random.default_rng(seed)
    return (r.standard_normal((n, R, K)).astype(np.float32), r.standard_normal((n, N, R)).astype(np.float32),
            r.random(n).astype(np.float32) + 0.5, ranks)


def test_oracle_by_scalar_loops():
    K, N, n, R, M = 32, 64, 3, 8, 5
    w, lo = _codes(K, N, 1), _lora(n, R, K, N, 2, np.array([8, 0, 3], np.int32))
    ids = np.array([2, -1, 0, 1, 3], np.int32)  # 3 is past the last adapter
    x = np.random.default_rng(3).standard_normal((M, K))
    W = O.dequant64(*w)
    want = np.zeros((M, N))
    for m in range(M):
        for c in range(N):
            v = sum(x[m, k] * W[k, c] for k in range(K))
            a = int(ids[m])
            if 0 <= a < n:
                for r in range(int(lo[3][a])):
                    v += float(lo[2][a]) * sum(x[m, k] * float(lo[0][a, r, k]) for k in range(K)) * float(lo[1][a, c, r])
            want[m, c] = v
    np.testing.assert_allclose(O.gemm_lora64(x, w, lo, ids), want, rtol=1e-12, atol=1e-12)


def test_oracle_closed_forms():
    K, N, M = 32, 64, 4
    w = _codes(K, N, 4)
    x = np.random.default_rng(5).standard_normal((M, K))
    ids = np.array([0, 1, 1, -1])
    a = np.zeros((2, 8, K), np.float32)
    a[:, 0, 3] = 1  # t = x[:, 3]
    b = np.zeros((2, N, 8), np.float32)
    b[1, :, 0] = 2
    y = O.gemm_lora64(x, w, (a, b, np.array([1, 0.5], np.float32), None), ids)
    base = O.gemm64(x, *w)
    np.testing.assert_array_equal(y[[0, 3]], base[[0, 3]])
    np.testing.assert_allclose(y[[1, 2]], base[[1, 2]] + x[[1, 2], 3:4], rtol=1e-13)
    # an MLP without adapters is the plain one
    g, u, d = _codes(K, N, 6), _codes(K, N, 7), _codes(N, K if K % 64 == 0 else 64, 8)
    d = _codes(N, 64, 8)
    h = O.silu64(O.gemm64(x, *g)) * O.gemm64(x, *u)
    np.testing.assert_array_equal(O.swiglu_mlp_lora64(x, g, u, d, None, None, None, ids), O.gemm64(h, *d))


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


def _desc(K, N, E=1):
    return L.WeightDesc(0x100000, 0x200000, K, N, 32, E, L.LAYOUT_GROUPED)


def _ldesc(a=0x300000, b=0x400000, scale=0x500000, ranks=None, rank=16, n=4):
    return L.LoraDesc(a, b, scale, ranks, rank, n)


def _p(v):
    return ctypes.c_void_p(v)


BAD_LORA = [(dict(a=0), L.ERR_INVALID_ARG), (dict(b=0), L.ERR_INVALID_ARG), (dict(scale=0), L.ERR_INVALID_ARG),
            (dict(a=0x300008), L.ERR_INVALID_ARG), (dict(b=0x400002), L.ERR_INVALID_ARG),
            (dict(scale=0x500004), L.ERR_INVALID_ARG), (dict(ranks=0x600004), L.ERR_INVALID_ARG),
            (dict(n=0), L.ERR_INVALID_ARG), (dict(rank=0), L.ERR_INVALID_ARG), (dict(rank=-8), L.ERR_INVALID_ARG),
            (dict(rank=12), L.ERR_UNSUPPORTED), (dict(rank=264), L.ERR_UNSUPPORTED)]


@pytest.mark.parametrize("bad,status", BAD_LORA)
def test_bad_adapters_are_refused(lib, bad, status):
    w, g, u, d = _desc(64, 128), _desc(64, 128), _desc(64, 128), _desc(128, 64)
    lo, ok = _ldesc(**bad), _ldesc()
    r = ctypes.byref
    assert lib.w4a16_gemm_lora_workspace_bytes(4, r(w), L.F32, r(lo)) == 0
    assert lib.w4a16_gemm_lora(_p(0x1000), L.F32, 4, r(w), r(lo), _p(0x2000), _p(0x8000), L.F32, _p(0x10000), 1 << 30,
                               None) == status
    for i in range(3):
        set_ = [ok, ok, ok]
        set_[i] = lo
        assert lib.w4a16_swiglu_mlp_lora_workspace_bytes(4, L.F32, r(g), r(u), r(d), *map(r, set_)) == 0
        assert lib.w4a16_swiglu_mlp_lora(_p(0x1000), L.F32, 4, r(g), r(u), r(d), *map(r, set_), _p(0x2000), _p(0x8000),
                                         L.F32, _p(0x10000), 1 << 30, None) == status


def test_gemm_lora_argument_checks(lib):
    w, lo = _desc(64, 128), _ldesc()
    r = ctypes.byref
    need = lib.w4a16_gemm_lora_workspace_bytes(4, r(w), L.BF16, r(lo))
    assert need > 0 and need % 256 == 0

    def call(x=0x1000, xt=L.BF16, M=4, w=w, lo=r(lo), ids=0x2000, y=0x8000, yt=L.F32, ws=0x10000, n=need):
        return lib.w4a16_gemm_lora(_p(x), xt, M, r(w), lo, _p(ids), _p(y), yt, _p(ws), n, None)

    assert call(M=0) == L.OK
    assert call(w=_desc(0, 128)) == L.OK and call(w=_desc(64, 0)) == L.OK
    assert call(M=-1) == L.ERR_INVALID_ARG
    assert call(xt=7) == L.ERR_INVALID_ARG and call(yt=7) == L.ERR_INVALID_ARG
    assert call(lo=None) == L.ERR_INVALID_ARG
    for arg in ("x", "ids", "y", "ws"):
        assert call(**{arg: 0}) == L.ERR_INVALID_ARG
        assert call(**{arg: 0x20008}) == L.ERR_INVALID_ARG  # misaligned
    assert call(y=0x1000) == L.ERR_INVALID_ARG  # y aliases x
    assert call(n=need - 1) == L.ERR_WORKSPACE
    assert call(w=_desc(64, 128, E=2)) == L.ERR_UNSUPPORTED
    assert call(w=_desc(64, 96)) == L.ERR_UNSUPPORTED
    assert lib.w4a16_gemm_lora_workspace_bytes(0, r(w), L.BF16, r(lo)) == 0
    assert lib.w4a16_gemm_lora_workspace_bytes(4, r(w), 7, r(lo)) == 0
    assert lib.w4a16_gemm_lora_workspace_bytes(4, r(w), L.BF16, None) == 0


def test_swiglu_mlp_lora_argument_checks(lib):
    g, u, d = _desc(64, 128), _desc(64, 128), _desc(128, 64)
    lo = _ldesc()
    r = ctypes.byref
    for have in range(8):  # any of the three may be absent
        set_ = [r(lo) if have >> i & 1 else None for i in range(3)]
        assert lib.w4a16_swiglu_mlp_lora_workspace_bytes(4, L.F32, r(g), r(u), r(d), *set_) > 0
    need = lib.w4a16_swiglu_mlp_lora_workspace_bytes(4, L.F32, r(g), r(u), r(d), r(lo), r(lo), r(lo))

    def call(x=0x1000, xt=L.F32, M=4, up=u, ids=0x2000, y=0x8000, yt=L.BF16, ws=0x10000, n=need):
        return lib.w4a16_swiglu_mlp_lora(_p(x), xt, M, r(g), r(up), r(d), r(lo), r(lo), r(lo), _p(ids), _p(y), yt,
                                         _p(ws), n, None)

    assert call(M=0) == L.OK
    assert call(M=-1) == L.ERR_INVALID_ARG
    assert call(xt=7) == L.ERR_INVALID_ARG and call(yt=7) == L.ERR_INVALID_ARG
    for arg in ("x", "ids", "y", "ws"):
        assert call(**{arg: 0}) == L.ERR_INVALID_ARG
        assert call(**{arg: 0x20008}) == L.ERR_INVALID_ARG
    assert call(y=0x1000) == L.ERR_INVALID_ARG
    assert call(n=need - 1) == L.ERR_WORKSPACE
    assert call(up=_desc(64, 192)) == L.ERR_UNSUPPORTED


def _w(K, N):
    return L.Weight(torch.zeros((1, K // 8, N), dtype=torch.int32), torch.zeros((1, K // 32, N)), K, N)


def _lo(n=3, R=8, K=64, N=128, **kw):
    t = dict(a=torch.zeros((n, R, K), dtype=torch.bfloat16), b=torch.zeros((n, N, R), dtype=torch.bfloat16),
             scale=torch.ones(n), ranks=None)
    t.update(kw)
    return L.Lora(**t)


@pytest.mark.parametrize("kw,err", [
    (dict(a=torch.zeros((3, 8, 64))), TypeError),                               # float32 adapters
    (dict(a=torch.zeros((8, 64), dtype=torch.bfloat16)), ValueError),           # one adapter, not a stack
    (dict(a=torch.zeros((3, 8, 32), dtype=torch.bfloat16)), ValueError),        # another K
    (dict(b=torch.zeros((3, 8, 128), dtype=torch.bfloat16)), ValueError),       # [n][R][N]
    (dict(b=torch.zeros((3, 8, 128), dtype=torch.bfloat16).transpose(1, 2)), ValueError),  # not contiguous
    (dict(scale=torch.ones(2)), ValueError),
    (dict(scale=torch.ones(3, dtype=torch.float64)), TypeError),
    (dict(ranks=torch.ones(3, dtype=torch.int64)), TypeError),
    (dict(), ValueError),                                                       # host tensors
])
def test_binding_rejects_bad_adapters(kw, err):
    ids, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(err):
        L.gemm_lora(torch.zeros((2, 64)), _w(64, 128), _lo(**kw), ids, torch.zeros((2, 128)), ws)


def test_binding_rejects_bad_ids_and_outputs(monkeypatch):
    monkeypatch.setattr(L, "_on_device", lambda **t: None)
    x, w, lo, ws = torch.zeros((2, 64)), _w(64, 128), _lo(), torch.zeros(256, dtype=torch.uint8)
    ids, y = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 128))
    with pytest.raises(TypeError):
        L.gemm_lora(x, w, lo, ids.long(), y, ws)
    with pytest.raises(ValueError):
        L.gemm_lora(x, w, lo, ids[:1], y, ws)
    with pytest.raises(TypeError):
        L.gemm_lora(x, w, lo, ids, y.half(), ws)
    with pytest.raises(ValueError):
        L.gemm_lora(x, w, lo, ids, y[:, :64], ws)
    with pytest.raises(ValueError):
        L.swiglu_mlp_lora(x, w, w, _w(128, 64), None, None, _lo(), ids, torch.zeros((2, 64)), ws)  # down is [128 -> 64]


@pytest.mark.parametrize("K,N", [(2 ** 26, 64), (64, 2 ** 26)])
def test_sizes_past_32_bit_row_bytes_are_refused(lib, K, N):
    r = ctypes.byref
    big, d, lo = _desc(K, N), _desc(N, K), _ldesc()
    assert lib.w4a16_gemm_lora_workspace_bytes(4, r(big), L.BF16, r(lo)) == 0
    assert lib.w4a16_gemm_lora(_p(0x1000), L.BF16, 4, r(big), r(lo), _p(0x2000), _p(0x8000), L.F32, _p(0x10000),
                               1 << 40, None) == L.ERR_UNSUPPORTED
    assert lib.w4a16_swiglu_mlp_lora_workspace_bytes(4, L.BF16, r(big), r(big), r(d), r(lo), None, None) == 0
    assert lib.w4a16_swiglu_mlp_lora(_p(0x1000), L.BF16, 4, r(big), r(big), r(d), r(lo), None, None, _p(0x2000),
                                     _p(0x8000), L.F32, _p(0x10000), 1 << 40, None) == L.ERR_UNSUPPORTED


@pytest.mark.parametrize("M", [1, 8, 9, 16, 17, 33, 64, 65, 513])
@pytest.mark.parametrize("xt", [L.F32, L.BF16])
def test_a_smaller_batch_needs_no_more_than_its_own_workspace(lib, M, xt):
    """The size is that of the call: exactly it is enough, one byte less is refused."""
    r = ctypes.byref
    w, lo = _desc(2048, 448), _ldesc()
    need = lib.w4a16_gemm_lora_workspace_bytes(M, r(w), xt, r(lo))
    assert need > 0 and need % 256 == 0
    assert lib.w4a16_gemm_lora(_p(0x1000), xt, M, r(w), r(lo), _p(0x2000), _p(0x800000), L.F32, _p(0x10000),
                               need - 1, None) == L.ERR_WORKSPACE
