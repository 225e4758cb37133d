"""CPU checks that the Python binding hands the library memory of the current device only:
weights, codes and scales too, on every compute call.  The tensors that are in order are
host tensors that answer as device ones, and the library must not be reached."""
import types

import pytest
import torch

import int4_w4a16_group_g32_amd as L

H, I, E, M, K_TOP = 64, 128, 4, 3, 2


class OnDevice(torch.Tensor):
    """A host tensor that says it is on device 0."""
    is_cuda = property(lambda self: True)
    index = 0

    def get_device(self):
        return self.index


class OnAnother(OnDevice):
    index = 1


def _t(shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


def _w(K, N, E=1):
    return L.Weight(_t((E, K // 32, N // 64, 64, 4), torch.int32), _t((E, K // 32, N)), K, N, E)


def _lora(K, N):
    return L.Lora(_t((2, 8, K), torch.bfloat16), _t((2, N, 8), torch.bfloat16), _t((2,)))


def _calls():
    """name -> (call, its tensors and weights by name)"""
    i32, u8 = torch.int32, torch.uint8
    dense = lambda: dict(gate=_w(H, I), up=_w(H, I), down=_w(I, H))  # noqa: E731
    stacks = lambda: dict(gate=_w(H, I, E), up=_w(H, I, E), down=_w(I, H, E))  # noqa: E731
    route = lambda: dict(topk_ids=_t((M, K_TOP), i32), topk_w=_t((M, K_TOP)))  # noqa: E731
    xy = lambda n=H: dict(x=_t((M, H)), y=_t((M, n)), ws=_t((256,), u8))  # noqa: E731
    static = dict(xy(), **dense())
    static.pop("ws")
    shared = dict(shared_gate=_w(H, I), shared_up=_w(H, I), shared_down=_w(I, H))
    decode = dict(xy(), logits=_t((M, E)), top_k=K_TOP, **stacks(), topk_ids=_t((M, K_TOP), i32),
                  topk_w=_t((M, K_TOP)))
    return {
        "gemm": (L.gemm, dict(xy(I), w=_w(H, I))),
        "swiglu_mlp": (L.swiglu_mlp, dict(xy(), **dense())),
        "swiglu_mlp_static": (L.swiglu_mlp_static, static),
        "gemm_lora": (L.gemm_lora, dict(xy(I), w=_w(H, I), lora=_lora(H, I), adapter_ids=_t((M,), i32))),
        "swiglu_mlp_lora": (L.swiglu_mlp_lora,
                            dict(xy(), **dense(), lora_gate=_lora(H, I), lora_up=_lora(H, I), lora_down=_lora(I, H),
                                 adapter_ids=_t((M,), i32))),
        "moe_grouped": (L.moe_grouped, dict(xy(), **route(), **stacks())),
        "moe_grouped_shared": (L.moe_grouped_shared, dict(xy(), **route(), **stacks(), **shared)),
        "moe_decode": (L.moe_decode, decode),
        "moe_decode_shared": (lambda **k: L.moe_decode(shared=(k.pop("sg"), k.pop("su"), k.pop("sd")), **k),
                              dict(decode, sg=_w(H, I), su=_w(H, I), sd=_w(I, H))),
        "moe_topk": (lambda **k: L.moe_topk(top_k=K_TOP, **k), dict(logits=_t((M, E)), **route())),
    }


class Reached(Exception):
    pass


def _reached():
    raise Reached


def _variants(args, change):
    """(what, arguments) with one tensor changed, the parts of weights and adapters among them."""
    for name, v in args.items():
        if isinstance(v, L.Weight):
            for part in ("qw", "scales"):
                w = L.Weight(v.qw, v.scales, v.K, v.N, v.num_experts)
                setattr(w, part, change(getattr(w, part)))
                yield f"{name}.{part}", dict(args, **{name: w})
        elif isinstance(v, L.Lora):
            for part in ("a", "b", "scale"):
                lo = L.Lora(v.a, v.b, v.scale)
                setattr(lo, part, change(getattr(lo, part)))
                yield f"{name}.{part}", dict(args, **{name: lo})
            yield f"{name}.ranks", dict(args, **{name: L.Lora(v.a, v.b, v.scale, change(_t((2,), torch.int32)))})
        elif isinstance(v, torch.Tensor):
            yield name, dict(args, **{name: change(v)})


def _refuses(name, change, monkeypatch, current=0):
    """The call goes through as it is, and refuses any one tensor changed."""
    monkeypatch.setattr(L, "load_library", _reached)
    monkeypatch.setattr(L, "_stream", lambda stream: 0)
    monkeypatch.setattr(L, "_current_device", lambda: current, raising=False)
    call, args = _calls()[name]
    with pytest.raises(Reached):
        call(**args)
    for what, bad in _variants(args, change):
        try:
            call(**bad)
        except ValueError:
            continue
        except Reached:
            pass
        pytest.fail(f"{name}: {what} went through")


@pytest.mark.parametrize("name", list(_calls()))
def test_host_memory_is_refused(name, monkeypatch):
    _refuses(name, lambda t: t.as_subclass(torch.Tensor), monkeypatch)


@pytest.mark.parametrize("name", list(_calls()))
def test_memory_of_another_device_is_refused(name, monkeypatch):
    _refuses(name, lambda t: t.as_subclass(OnAnother), monkeypatch)


@pytest.mark.parametrize("name", list(_calls()))
def test_a_device_that_is_not_current_is_refused(name, monkeypatch):
    monkeypatch.setattr(L, "load_library", _reached)
    monkeypatch.setattr(L, "_stream", lambda stream: 0)
    monkeypatch.setattr(L, "_current_device", lambda: 1, raising=False)
    call, args = _calls()[name]
    with pytest.raises(ValueError):
        call(**args)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(L, "_current_device", lambda: 1, raising=False)
    of = lambda d: types.SimpleNamespace(device_index=d, cuda_stream=0x70)  # noqa: E731
    assert L._stream(of(1)) == 0x70
    with pytest.raises(ValueError):
        L._stream(of(0))
