"""CPU checks of w4a16_moe_decode: every refusal of the C entry point and of the
binding (nothing is enqueued: the pointers are not device memory)."""
import ctypes

import pytest
import torch

import int4_w4a16_group_g32_amd as L


@pytest.fixture(scope="module")
def lib():
    return L.load_library()


def _desc(K, N, E=6, group=32, layout=L.LAYOUT_GROUPED, qw=0x100000):
    return L.WeightDesc(qw, 0x200000, K, N, group, E, layout)


def _p(v):
    return ctypes.c_void_p(v)


def _r(d):
    return None if d is None else ctypes.byref(d)


STACK = (_desc(64, 128), _desc(64, 128), _desc(128, 64))
ONE = (_desc(64, 128, 1), _desc(64, 128, 1), _desc(128, 64, 1))
NONE = (None, None, None)


def _need(lib, M=4, k=2, xt=L.F32, stack=STACK, shared=NONE):
    return lib.w4a16_moe_decode_workspace_bytes(M, k, xt, *map(_r, stack), *map(_r, shared))


def _call(lib, x=0x1000, xt=L.F32, M=4, logits=0x2000, k=2, stack=STACK, shared=NONE, ids=None, w=None, y=0x8000,
          yt=L.F32, ws=0x10000, n=1 << 30):
    return lib.w4a16_moe_decode(_p(x), xt, M, _p(logits), k, *map(_r, stack), *map(_r, shared), _p(ids), _p(w), _p(y),
                                yt, _p(ws), n, None)


def test_argument_checks(lib):
    need = _need(lib)
    assert need > 0 and need % 256 == 0
    assert _need(lib, shared=ONE) > need
    assert _call(lib, M=0) == L.OK
    assert _call(lib, M=-1) == L.ERR_INVALID_ARG
    assert _call(lib, k=0) == L.ERR_INVALID_ARG and _call(lib, k=7) == L.ERR_INVALID_ARG
    assert _call(lib, xt=7) == L.ERR_INVALID_ARG and _call(lib, yt=7) == L.ERR_INVALID_ARG
    for arg in ("x", "logits", "y", "ws"):
        assert _call(lib, **{arg: 0}) == L.ERR_INVALID_ARG
        assert _call(lib, **{arg: 0x20008}) == L.ERR_INVALID_ARG
    assert _call(lib, ids=0x3004) == L.ERR_INVALID_ARG and _call(lib, w=0x3008) == L.ERR_INVALID_ARG
    assert _call(lib, y=0x1000) == L.ERR_INVALID_ARG
    assert _call(lib, n=need - 1) == L.ERR_WORKSPACE
    assert _need(lib, M=0) == 0 and _need(lib, k=0) == 0 and _need(lib, xt=7) == 0


def test_limits(lib):
    assert _need(lib, M=8) > 0 and _need(lib, M=9) == 0
    assert _need(lib, M=16, xt=L.BF16) > 0 and _need(lib, M=17, xt=L.BF16) == 0
    assert _call(lib, M=9) == L.ERR_UNSUPPORTED and _call(lib, M=17, xt=L.BF16) == L.ERR_UNSUPPORTED
    for E, k, ok in ((1024, 32, True), (1025, 2, False), (64, 33, False)):
        stack = (_desc(64, 128, E), _desc(64, 128, E), _desc(128, 64, E))
        assert (_need(lib, k=k, stack=stack) > 0) == ok
        if not ok:
            assert _call(lib, k=k, stack=stack) == L.ERR_UNSUPPORTED


@pytest.mark.parametrize("stack,shared,status", [
    ((_desc(64, 128), _desc(64, 128), _desc(128, 64, 5)), NONE, L.ERR_UNSUPPORTED),
    ((_desc(64, 128), _desc(64, 192), _desc(128, 64)), NONE, L.ERR_UNSUPPORTED),
    ((_desc(64, 128), _desc(64, 128, group=64), _desc(128, 64)), NONE, L.ERR_UNSUPPORTED),
    ((_desc(64, 128), _desc(64, 128), _desc(128, 128)), NONE, L.ERR_UNSUPPORTED),
    ((_desc(64, 128), _desc(64, 128), _desc(128, 64, layout=L.LAYOUT_CANONICAL)), NONE, L.ERR_UNSUPPORTED),
    ((_desc(64, 128, qw=0), _desc(64, 128), _desc(128, 64)), NONE, L.ERR_INVALID_ARG),
    (STACK, (ONE[0], ONE[1], None), L.ERR_INVALID_ARG),
    (STACK, (None, None, ONE[2]), L.ERR_INVALID_ARG),
    (STACK, STACK, L.ERR_UNSUPPORTED),  # a shared expert is one
    (STACK, (_desc(64, 192, 1), _desc(64, 192, 1), _desc(192, 64, 1)), L.ERR_UNSUPPORTED),
    (STACK, (ONE[0], ONE[1], _desc(128, 64, 1, 64)), L.ERR_UNSUPPORTED),
])
def test_weights_that_do_not_fit_are_refused(lib, stack, shared, status):
    assert _need(lib, stack=stack, shared=shared) == 0
    assert _call(lib, stack=stack, shared=shared) == status


def _w(K, N, E):
    return L.Weight(torch.zeros((E, K // 8, N), dtype=torch.int32), torch.zeros((E, K // 32, N)), K, N, E)


def test_binding_rejects_bad_tensors(monkeypatch):
    g, u, d = _w(64, 128, 4), _w(64, 128, 4), _w(128, 64, 4)
    x, lg, y, ws = torch.zeros((3, 64)), torch.zeros((3, 4)), torch.zeros((3, 64)), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):  # host tensors
        L.moe_decode(x, lg, 2, g, u, d, y, ws)
    monkeypatch.setattr(L, "_on_device", lambda **t: None)
    for kw, err in ((dict(logits=lg.double()), TypeError), (dict(logits=lg[:2]), ValueError),
                    (dict(logits=torch.zeros((3, 5))), ValueError), (dict(x=x.half()), TypeError),
                    (dict(x=torch.zeros((3, 32))), ValueError), (dict(y=torch.zeros((3, 128))), ValueError),
                    (dict(y=y.half()), TypeError), (dict(ws=torch.zeros(64)), TypeError),
                    (dict(topk_ids=torch.zeros((3, 2), dtype=torch.int64)), TypeError),
                    (dict(topk_ids=torch.zeros((3, 3), dtype=torch.int32)), ValueError),
                    (dict(topk_w=torch.zeros((2, 2))), ValueError)):
        args = dict(x=x, logits=lg, top_k=2, gate=g, up=u, down=d, y=y, ws=ws)
        args.update(kw)
        with pytest.raises(err):
            L.moe_decode(**args)
