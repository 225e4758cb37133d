"""Python binding of libw4a16.so, the MI355X (gfx950) W4A16 group-32 library.

Argument marshalling only: every computation runs in the HIP kernels behind
the C ABI declared in include/w4a16.h.  PyTorch supplies device memory and
streams.  There is no fallback: if the library is not built, importing a
compute function raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libw4a16.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = range(5)
F32, BF16 = 0, 1
MXFP4 = 2  # activations given as an MxMatrix (the binding's own code, not the library's)
MX_ROWS, MX_TILED = 0, 1
LAYOUT_CANONICAL, LAYOUT_GROUPED = 0, 1
GROUP = 32

# every symbol include/w4a16.h declares
EXPORTS = (
    "w4a16_status_string",
    "w4a16_workspace_init",
    "w4a16_quantize",
    "w4a16_quantize_group",
    "w4a16_prepacked_bytes",
    "w4a16_prepack",
    "w4a16_dequantize",
    "w4a16_gemm_workspace_bytes",
    "w4a16_gemm",
    "w4a16_gemm_timed",
    "w4a16_swiglu_mlp_workspace_bytes",
    "w4a16_swiglu_mlp",
    "w4a16_swiglu_mlp_timed",
    "w4a16_swiglu_mlp_static",
    "w4a16_gemm_lora_workspace_bytes",
    "w4a16_gemm_lora",
    "w4a16_swiglu_mlp_lora_workspace_bytes",
    "w4a16_swiglu_mlp_lora",
    "w4a16_moe_topk",
    "w4a16_moe_route",
    "w4a16_moe_workspace_bytes",
    "w4a16_moe_grouped",
    "w4a16_moe_shared_workspace_bytes",
    "w4a16_moe_grouped_shared",
    "w4a16_moe_decode_workspace_bytes",
    "w4a16_moe_decode",
    "w4a16_moe_grouped_timed",
    "w4a16_mx_codes_bytes",
    "w4a16_mx_scales_bytes",
    "w4a16_mx_quantize",
    "w4a16_mx_quantize_weight",
    "w4a16_mx_prepack",
    "w4a16_mx_dequantize",
    "w4a16_mx_gemm_workspace_bytes",
    "w4a16_mx_gemm",
    "w4a16_mx_gemm_a4_workspace_bytes",
    "w4a16_mx_gemm_a4",
    "w4a16_mx_swiglu_mlp_workspace_bytes",
    "w4a16_mx_swiglu_mlp",
    "w4a16_mx_swiglu_mlp_a4_workspace_bytes",
    "w4a16_mx_swiglu_mlp_a4",
    "w4a16_block_norm",
)


class W4A16Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


class WeightDesc(ctypes.Structure):
    _fields_ = [
        ("qw", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("K", ctypes.c_int32),
        ("N", ctypes.c_int32),
        ("group_size", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("layout", ctypes.c_int32),
    ]


class LoraDesc(ctypes.Structure):
    _fields_ = [
        ("a", ctypes.c_void_p),
        ("b", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("ranks", ctypes.c_void_p),
        ("rank", ctypes.c_int32),
        ("num_adapters", ctypes.c_int32),
    ]


class MxDesc(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("rows", ctypes.c_int32),
        ("K", ctypes.c_int32),
        ("layout", ctypes.c_int32),
    ]


class NormDesc(ctypes.Structure):
    _fields_ = [
        ("y", ctypes.c_void_p),
        ("r", ctypes.c_void_p),
        ("r_out", ctypes.c_void_p),
        ("post_w", ctypes.c_void_p),
        ("pre_w", ctypes.c_void_p),
        ("gate", ctypes.c_void_p),
        ("gate_rows", ctypes.c_int32),
        ("n", ctypes.c_void_p),
        ("n_codes", ctypes.c_void_p),
        ("n_scales", ctypes.c_void_p),
        ("y_type", ctypes.c_int32),
        ("r_type", ctypes.c_int32),
        ("w_type", ctypes.c_int32),
        ("n_type", ctypes.c_int32),
        ("alpha", ctypes.c_double),
        ("eps", ctypes.c_double),
    ]


_lib = None


def load_library() -> ctypes.CDLL:
    """Load libw4a16.so (built in-tree by int4_w4a16_group_g32_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m int4_w4a16_group_g32_amd.build`")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        dp = ctypes.POINTER(WeightDesc)
        lp = ctypes.POINTER(LoraDesc)
        mp = ctypes.POINTER(MxDesc)
        sig = {
            "w4a16_status_string": (ctypes.c_char_p, [i32]),
            "w4a16_workspace_init": (i32, [vp, sz, vp]),
            "w4a16_quantize": (i32, [vp, i32, i32, i32, vp, sz, vp, sz, vp]),
            "w4a16_quantize_group": (i32, [vp, i32, i32, i32, i32, vp, sz, vp, sz, vp]),
            "w4a16_prepacked_bytes": (sz, [dp]),
            "w4a16_prepack": (i32, [dp, vp, sz, dp, vp]),
            "w4a16_dequantize": (i32, [dp, vp, sz, vp]),
            "w4a16_gemm_workspace_bytes": (sz, [i32, dp, i32]),
            "w4a16_gemm": (i32, [vp, i32, i32, dp, vp, vp, sz, vp]),
            "w4a16_gemm_timed": (i32, [vp, i32, i32, dp, vp, vp, sz, vp, vp, i32, ctypes.POINTER(i32)]),
            "w4a16_swiglu_mlp_workspace_bytes": (sz, [i32, i32, dp, dp, dp]),
            "w4a16_swiglu_mlp": (i32, [vp, i32, i32, dp, dp, dp, vp, vp, sz, vp]),
            "w4a16_swiglu_mlp_timed": (i32, [vp, i32, i32, dp, dp, dp, vp, vp, sz, vp, vp, i32,
                                             ctypes.POINTER(i32)]),
            "w4a16_swiglu_mlp_static": (i32, [vp, i32, i32, dp, dp, dp, vp, vp]),
            "w4a16_gemm_lora_workspace_bytes": (sz, [i32, dp, i32, lp]),
            "w4a16_gemm_lora": (i32, [vp, i32, i32, dp, lp, vp, vp, i32, vp, sz, vp]),
            "w4a16_swiglu_mlp_lora_workspace_bytes": (sz, [i32, i32, dp, dp, dp, lp, lp, lp]),
            "w4a16_swiglu_mlp_lora": (i32, [vp, i32, i32, dp, dp, dp, lp, lp, lp, vp, vp, i32, vp, sz, vp]),
            "w4a16_moe_topk": (i32, [vp, i32, i32, i32, vp, vp, vp]),
            "w4a16_moe_route": (i32, [vp, i32, i32, i32, vp, vp, vp, vp, vp]),
            "w4a16_moe_workspace_bytes": (sz, [i32, i32, i32, dp, dp, dp]),
            "w4a16_moe_grouped": (i32, [vp, i32, i32, vp, vp, i32, dp, dp, dp, vp, vp, sz, vp]),
            "w4a16_moe_shared_workspace_bytes": (sz, [i32, i32, i32, dp, dp, dp, dp, dp, dp]),
            "w4a16_moe_grouped_shared": (i32, [vp, i32, i32, vp, vp, i32, dp, dp, dp, dp, dp, dp, vp, vp, sz,
                                               vp]),
            "w4a16_moe_decode_workspace_bytes": (sz, [i32, i32, i32, dp, dp, dp, dp, dp, dp]),
            "w4a16_moe_decode": (i32, [vp, i32, i32, vp, i32, dp, dp, dp, dp, dp, dp, vp, vp, vp, i32, vp, sz, vp]),
            "w4a16_moe_grouped_timed": (i32, [vp, i32, i32, vp, vp, i32, dp, dp, dp, vp, vp, sz, vp, vp,
                                              i32, ctypes.POINTER(i32)]),
            "w4a16_mx_codes_bytes": (sz, [i32, i32, i32]),
            "w4a16_mx_scales_bytes": (sz, [i32, i32, i32]),
            "w4a16_mx_quantize": (i32, [vp, i32, i32, i32, vp, sz, vp, sz, vp]),
            "w4a16_mx_quantize_weight": (i32, [vp, i32, i32, i32, vp, sz, vp, sz, vp]),
            "w4a16_mx_prepack": (i32, [mp, vp, sz, vp, sz, mp, vp]),
            "w4a16_mx_dequantize": (i32, [mp, vp, i32, sz, vp]),
            "w4a16_mx_gemm_workspace_bytes": (sz, [i32, i32, mp]),
            "w4a16_mx_gemm": (i32, [vp, i32, i32, mp, vp, i32, vp, sz, vp]),
            "w4a16_mx_gemm_a4_workspace_bytes": (sz, [i32, mp]),
            "w4a16_mx_gemm_a4": (i32, [mp, mp, vp, i32, vp, sz, vp]),
            "w4a16_mx_swiglu_mlp_workspace_bytes": (sz, [i32, i32, mp, mp, mp]),
            "w4a16_mx_swiglu_mlp": (i32, [vp, i32, i32, mp, mp, mp, vp, i32, vp, sz, vp]),
            "w4a16_mx_swiglu_mlp_a4_workspace_bytes": (sz, [i32, mp, mp, mp]),
            "w4a16_mx_swiglu_mlp_a4": (i32, [mp, mp, mp, mp, vp, i32, vp, sz, vp]),
            "w4a16_block_norm": (i32, [ctypes.POINTER(NormDesc), i32, i32, vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load_library().w4a16_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != OK:
        raise W4A16Error(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()  # (the signatures' c_void_p takes an int)


def _stream(stream):
    if stream is None:  # the current stream's handle, without a Stream object around it (0.4 us for 2.9)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if stream.device_index != _current_device():
        raise ValueError(f"stream is of device {stream.device_index}, the current device is {_current_device()}")
    return stream.cuda_stream


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype == torch.float32:
        return F32
    if x.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"activations must be float32 or bfloat16, got {x.dtype}")


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _need(t: torch.Tensor, name: str, dtype, shape=None):
    """Check a tensor handed to the library: dtype, contiguity and shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _on_device(**tensors):
    """Every tensor the library reads or writes, a Weight's codes and scales too, must be memory of the
    current device: the calls launch there, on one of its streams."""
    dev = None
    for name, v in tensors.items():
        for t in (v.qw, v.scales) if isinstance(v, Weight) else (v.codes, v.scales) if isinstance(v, MxMatrix) else (v,):
            if not isinstance(t, torch.Tensor):
                continue
            d = t.get_device()
            if d == dev:
                continue
            if d < 0:
                raise ValueError(f"{name} must be a device tensor, got {t.device}")
            dev = _current_device()
            if d != dev:
                raise ValueError(f"{name} is on device {d}, the current device is {dev}")


# The MXFP4 calls and block_norm ask of each tensor what `_need` and `_on_device` ask, in one expression
# (0.3 us for 1.1: a few-row call is bound by the host); those two then say what is wrong.
_F32, _BF16, _U8 = torch.float32, torch.bfloat16, torch.uint8


def _fits(t, dtype, shape, dev: int) -> bool:
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev


def _ready(t, name: str, dtype, shape, dev: int):
    """Refuses a tensor of another type, shape, layout or device than the current one, `dev`."""
    if not (isinstance(t, torch.Tensor) and _fits(t, dtype, shape, dev)):
        _need(t, name, dtype, shape)
        _on_device(**{name: t})


def _device_of(t, name: str = "y") -> int:
    """The current device, of which `t` must be."""
    try:
        d = t.get_device()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    return d if d >= 0 and d == _current_device() else -2  # (no tensor is of device -2)


def _stream_of(stream, dev: int):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _need_x(x: torch.Tensor, K: int):
    _dtype_code(x)
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"activations must be [M][{K}], got {tuple(x.shape)}")
    _need(x, "x", x.dtype)


@dataclass
class Weight:
    """A W4A16 weight (or expert stack): codes, scales and their shape."""
    qw: torch.Tensor          # int32, CANONICAL [E][K/8][N] or GROUPED [E][K/32][N][4]
    scales: torch.Tensor      # float32 [E][K/group_size][N]
    K: int
    N: int
    num_experts: int = 1
    layout: int = LAYOUT_GROUPED
    group_size: int = GROUP   # rows per scale: 32, 64 or 128

    def desc(self) -> WeightDesc:
        return WeightDesc(self.qw.data_ptr(), self.scales.data_ptr(), self.K, self.N, self.group_size,
                          self.num_experts, self.layout)


@dataclass
class MxMatrix:
    """An MXFP4 matrix of `rows` rows of K values: activations, or a weight's output columns."""
    codes: torch.Tensor   # uint8, ROWS [rows][K/2] or TILED
    scales: torch.Tensor  # uint8, ROWS [rows][K/32] or TILED
    rows: int
    K: int
    layout: int = MX_ROWS

    def desc(self) -> MxDesc:
        return MxDesc(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.K, self.layout)

    def check(self, name: str):
        """The tensors' dtypes, sizes and devices for the shape."""
        self._ready(name, _device_of(self.codes) if isinstance(self.codes, torch.Tensor) else -2)

    def _ready(self, name: str, dev: int):
        c, s, rows, K = self.codes, self.scales, self.rows, self.K
        if self.layout == MX_TILED:
            tiles = -(-rows // 64) * -(-K // 128)
            nc, ns = tiles * 4096, tiles * 256
        else:
            nc, ns = rows * (K // 2), rows * (K // 32)
        try:
            if (c.dtype is _U8 and s.dtype is _U8 and c.numel() == nc and s.numel() == ns and c.is_contiguous()
                    and s.is_contiguous() and c.get_device() == dev and s.get_device() == dev):
                return
        except AttributeError:  # (no tensor)
            pass
        _need(c, f"{name}.codes", torch.uint8)
        _need(s, f"{name}.scales", torch.uint8)
        if (c.numel(), s.numel()) != (nc, ns):
            raise ValueError(f"{name}: codes and scales must have {nc} and {ns} bytes for {rows} rows of {K}, got "
                             f"{c.numel()} and {s.numel()}")
        _on_device(**{name: self})


@dataclass
class Lora:
    """The adapters of one projection [K -> N], one stack for all requests."""
    a: torch.Tensor                     # bfloat16 [n][R][K]
    b: torch.Tensor                     # bfloat16 [n][N][R]
    scale: torch.Tensor                 # float32 [n]
    ranks: torch.Tensor | None = None   # int32 [n]: ranks in use (None: R)

    def desc(self) -> LoraDesc:
        return LoraDesc(self.a.data_ptr(), self.b.data_ptr(), self.scale.data_ptr(),
                        None if self.ranks is None else self.ranks.data_ptr(), self.a.shape[1], self.a.shape[0])

    def check(self, K: int, N: int):
        """The stack's dtypes, shapes and devices for a projection [K -> N]."""
        if not isinstance(self.a, torch.Tensor) or self.a.dim() != 3:
            raise ValueError("lora.a must be [num_adapters][rank][K]")
        n, R, _ = self.a.shape
        _need(self.a, "lora.a", torch.bfloat16, (n, R, K))
        _need(self.b, "lora.b", torch.bfloat16, (n, N, R))
        _need(self.scale, "lora.scale", torch.float32, (n,))
        if self.ranks is not None:
            _need(self.ranks, "lora.ranks", torch.int32, (n,))
        _on_device(lora_a=self.a, lora_b=self.b, lora_scale=self.scale, lora_ranks=self.ranks)


def _lref(lora):
    return None if lora is None else ctypes.byref(lora.desc())


def _dref(w):
    return None if w is None else ctypes.byref(w.desc() if isinstance(w, Weight) else w)


# ---------------------------------------------------------------- format

def workspace_init(ws: torch.Tensor, stream=None):
    _on_device(ws=ws)
    _check(load_library().w4a16_workspace_init(_ptr(ws), ws.numel() * ws.element_size(),
                                                _stream(stream)), "w4a16_workspace_init")


def quantize(w: torch.Tensor, qw: torch.Tensor, scales: torch.Tensor, stream=None, group_size: int = GROUP):
    """w float32 [E][K][N] (or [K][N]) -> CANONICAL qw, scales [E][K/group_size][N] (caller-allocated)."""
    _need(w, "w", torch.float32)
    _need(qw, "qw", torch.int32)
    _need(scales, "scales", torch.float32)
    _on_device(w=w, qw=qw, scales=scales)
    E = 1 if w.dim() == 2 else w.shape[0]
    K, N = w.shape[-2], w.shape[-1]
    if group_size == GROUP:
        st = load_library().w4a16_quantize(_ptr(w), K, N, E, _ptr(qw), _nbytes(qw), _ptr(scales), _nbytes(scales),
                                           _stream(stream))
    else:
        st = load_library().w4a16_quantize_group(_ptr(w), K, N, E, group_size, _ptr(qw), _nbytes(qw),
                                                 _ptr(scales), _nbytes(scales), _stream(stream))
    _check(st, "w4a16_quantize")


def prepacked_bytes(src: Weight) -> int:
    """Bytes of GROUPED codes w4a16_prepack writes for `src` (0 for an unsupported descriptor)."""
    return load_library().w4a16_prepacked_bytes(_dref(src))


def prepack(src: Weight, dst_qw: torch.Tensor, stream=None) -> Weight:
    _need(dst_qw, "dst_qw", torch.int32)
    _on_device(dst_qw=dst_qw, qw=src.qw, scales=src.scales)
    out = WeightDesc()
    _check(load_library().w4a16_prepack(_dref(src), _ptr(dst_qw), _nbytes(dst_qw), ctypes.byref(out),
                                        _stream(stream)), "w4a16_prepack")
    return Weight(dst_qw, src.scales, out.K, out.N, out.num_experts, out.layout, out.group_size)


def dequantize(w: Weight, out: torch.Tensor, stream=None):
    _need(out, "out", torch.float32)
    _on_device(out=out, qw=w.qw, scales=w.scales)
    _check(load_library().w4a16_dequantize(_dref(w), _ptr(out), _nbytes(out), _stream(stream)), "w4a16_dequantize")


# ---------------------------------------------------------------- compute

def gemm_workspace_bytes(M: int, w: Weight, xt: int) -> int:
    return load_library().w4a16_gemm_workspace_bytes(M, _dref(w), xt)


def gemm(x: torch.Tensor, w: Weight, y: torch.Tensor, ws: torch.Tensor, stream=None):
    _need_x(x, w.K)
    _need(y, "y", torch.float32, (x.shape[0], w.N))
    _need(ws, "ws", torch.uint8)
    _on_device(x=x, w=w, y=y, ws=ws)
    _check(load_library().w4a16_gemm(_ptr(x), _dtype_code(x), x.shape[0], _dref(w), _ptr(y), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)), "w4a16_gemm")


def swiglu_mlp_workspace_bytes(M: int, xt: int, gate: Weight, up: Weight, down: Weight) -> int:
    return load_library().w4a16_swiglu_mlp_workspace_bytes(M, xt, _dref(gate), _dref(up), _dref(down))


def swiglu_mlp(x: torch.Tensor, gate: Weight, up: Weight, down: Weight, y: torch.Tensor,
               ws: torch.Tensor, stream=None):
    _need_x(x, gate.K)
    _need(y, "y", torch.float32, (x.shape[0], down.N))
    _need(ws, "ws", torch.uint8)
    _on_device(x=x, gate=gate, up=up, down=down, y=y, ws=ws)
    _check(load_library().w4a16_swiglu_mlp(_ptr(x), _dtype_code(x), x.shape[0], _dref(gate), _dref(up),
                                           _dref(down), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                                           _stream(stream)), "w4a16_swiglu_mlp")


def swiglu_mlp_static(x: torch.Tensor, gate: Weight, up: Weight, down: Weight, y: torch.Tensor, stream=None):
    """swiglu_mlp on the library's static per-GPU scratch (no workspace, no allocation)."""
    _need_x(x, gate.K)
    _need(y, "y", torch.float32, (x.shape[0], down.N))
    _on_device(x=x, gate=gate, up=up, down=down, y=y)
    _check(load_library().w4a16_swiglu_mlp_static(_ptr(x), _dtype_code(x), x.shape[0], _dref(gate), _dref(up),
                                                  _dref(down), _ptr(y), _stream(stream)), "w4a16_swiglu_mlp_static")


def _need_y(y, shape) -> int:
    """y float32 or bfloat16 of this shape; returns its dtype code."""
    yt = _dtype_code(y)
    _need(y, "y", y.dtype, shape)
    return yt


def _need_ids(adapter_ids, M: int):
    _need(adapter_ids, "adapter_ids", torch.int32, (M,))
    _on_device(adapter_ids=adapter_ids)


def gemm_lora_workspace_bytes(M: int, w: Weight, xt: int, lora: Lora) -> int:
    return load_library().w4a16_gemm_lora_workspace_bytes(M, _dref(w), xt, _lref(lora))


def gemm_lora(x: torch.Tensor, w: Weight, lora: Lora, adapter_ids: torch.Tensor, y: torch.Tensor, ws: torch.Tensor,
              stream=None):
    """gemm plus each row's low-rank adapter (adapter_ids int32 [M], -1: none); y float32 or bfloat16."""
    _need_x(x, w.K)
    lora.check(w.K, w.N)
    _need_ids(adapter_ids, x.shape[0])
    yt = _need_y(y, (x.shape[0], w.N))
    _need(ws, "ws", torch.uint8)
    _on_device(x=x, w=w, y=y, ws=ws)
    _check(load_library().w4a16_gemm_lora(_ptr(x), _dtype_code(x), x.shape[0], _dref(w), _lref(lora),
                                          _ptr(adapter_ids), _ptr(y), yt, _ptr(ws), _nbytes(ws), _stream(stream)),
           "w4a16_gemm_lora")


def swiglu_mlp_lora_workspace_bytes(M: int, xt: int, gate: Weight, up: Weight, down: Weight, lora_gate: Lora | None,
                                    lora_up: Lora | None, lora_down: Lora | None) -> int:
    return load_library().w4a16_swiglu_mlp_lora_workspace_bytes(M, xt, _dref(gate), _dref(up), _dref(down),
                                                                _lref(lora_gate), _lref(lora_up), _lref(lora_down))


def swiglu_mlp_lora(x: torch.Tensor, gate: Weight, up: Weight, down: Weight, lora_gate: Lora | None,
                    lora_up: Lora | None, lora_down: Lora | None, adapter_ids: torch.Tensor, y: torch.Tensor,
                    ws: torch.Tensor, stream=None):
    """swiglu_mlp plus each row's low-rank adapters on any of the three projections (None: no adapters there)."""
    _need_x(x, gate.K)
    for lora, w in ((lora_gate, gate), (lora_up, up), (lora_down, down)):
        if lora is not None:
            lora.check(w.K, w.N)
    _need_ids(adapter_ids, x.shape[0])
    yt = _need_y(y, (x.shape[0], down.N))
    _need(ws, "ws", torch.uint8)
    _on_device(x=x, gate=gate, up=up, down=down, y=y, ws=ws)
    _check(load_library().w4a16_swiglu_mlp_lora(_ptr(x), _dtype_code(x), x.shape[0], _dref(gate), _dref(up),
                                                _dref(down), _lref(lora_gate), _lref(lora_up), _lref(lora_down),
                                                _ptr(adapter_ids), _ptr(y), yt, _ptr(ws), _nbytes(ws),
                                                _stream(stream)), "w4a16_swiglu_mlp_lora")


def moe_topk(logits: torch.Tensor, top_k: int, topk_ids: torch.Tensor, topk_w: torch.Tensor, stream=None):
    """Top-k experts per token row of float32 logits [M][E] and their softmax gate weights."""
    _need(logits, "logits", torch.float32)
    M, E = logits.shape
    _need(topk_ids, "topk_ids", torch.int32, (M, top_k))
    _need(topk_w, "topk_w", torch.float32, (M, top_k))
    _on_device(logits=logits, topk_ids=topk_ids, topk_w=topk_w)
    _check(load_library().w4a16_moe_topk(_ptr(logits), M, E, top_k, _ptr(topk_ids), _ptr(topk_w),
                                         _stream(stream)), "w4a16_moe_topk")


def moe_route(topk_ids: torch.Tensor, num_experts: int, counts, offsets, sorted_pairs, inv, stream=None):
    _need(topk_ids, "topk_ids", torch.int32)
    M, k = topk_ids.shape
    _need(counts, "counts", torch.int32, (num_experts,))
    _need(offsets, "offsets", torch.int32, (num_experts + 1,))
    for t, name in ((sorted_pairs, "sorted_pairs"), (inv, "inv")):
        _need(t, name, torch.int32)
        if t.numel() < M * k:
            raise ValueError(f"{name} must hold at least {M * k} entries")
    _on_device(topk_ids=topk_ids, counts=counts, offsets=offsets, sorted_pairs=sorted_pairs, inv=inv)
    _check(load_library().w4a16_moe_route(_ptr(topk_ids), M, k, num_experts, _ptr(counts), _ptr(offsets),
                                          _ptr(sorted_pairs), _ptr(inv), _stream(stream)), "w4a16_moe_route")


def moe_workspace_bytes(M: int, top_k: int, xt: int, gate: Weight, up: Weight, down: Weight) -> int:
    return load_library().w4a16_moe_workspace_bytes(M, top_k, xt, _dref(gate), _dref(up), _dref(down))


def moe_shared_workspace_bytes(M: int, top_k: int, xt: int, gate: Weight, up: Weight, down: Weight,
                               shared_gate: Weight, shared_up: Weight, shared_down: Weight) -> int:
    return load_library().w4a16_moe_shared_workspace_bytes(M, top_k, xt, _dref(gate), _dref(up), _dref(down),
                                                           _dref(shared_gate), _dref(shared_up),
                                                           _dref(shared_down))


def _check_moe_args(x, topk_ids, topk_w, gate: Weight, up: Weight, down: Weight, y, ws):
    """topk_ids int32 [M][k] (torch.topk's int64 ids must be converted), topk_w
    float32 [M][k], x [M][H], y float32 [M][H]; returns (M, k)."""
    _need(topk_ids, "topk_ids", torch.int32)
    if topk_ids.dim() != 2:
        raise ValueError(f"topk_ids must be [M][top_k], got {tuple(topk_ids.shape)}")
    M, k = topk_ids.shape
    _need(topk_w, "topk_w", torch.float32, (M, k))
    _need_x(x, gate.K)
    if x.shape[0] != M:
        raise ValueError(f"x has {x.shape[0]} rows, topk_ids {M}")
    _need(y, "y", torch.float32, (M, down.N))
    _need(ws, "ws", torch.uint8)
    _on_device(x=x, topk_ids=topk_ids, topk_w=topk_w, gate=gate, up=up, down=down, y=y, ws=ws)
    return M, k


def moe_grouped_shared(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, gate: Weight, up: Weight,
                       down: Weight, shared_gate: Weight, shared_up: Weight, shared_down: Weight, y: torch.Tensor,
                       ws: torch.Tensor, stream=None):
    M, k = _check_moe_args(x, topk_ids, topk_w, gate, up, down, y, ws)
    _on_device(shared_gate=shared_gate, shared_up=shared_up, shared_down=shared_down)
    _check(load_library().w4a16_moe_grouped_shared(_ptr(x), _dtype_code(x), M, _ptr(topk_ids), _ptr(topk_w), k,
                                                   _dref(gate), _dref(up), _dref(down), _dref(shared_gate),
                                                   _dref(shared_up), _dref(shared_down), _ptr(y), _ptr(ws),
                                                   ws.numel() * ws.element_size(), _stream(stream)),
           "w4a16_moe_grouped_shared")


def moe_grouped(x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, gate: Weight, up: Weight,
                down: Weight, y: torch.Tensor, ws: torch.Tensor, stream=None):
    M, k = _check_moe_args(x, topk_ids, topk_w, gate, up, down, y, ws)
    _check(load_library().w4a16_moe_grouped(_ptr(x), _dtype_code(x), M, _ptr(topk_ids), _ptr(topk_w), k,
                                            _dref(gate), _dref(up), _dref(down), _ptr(y), _ptr(ws),
                                            ws.numel() * ws.element_size(), _stream(stream)),
           "w4a16_moe_grouped")


def moe_decode_workspace_bytes(M: int, top_k: int, xt: int, gate: Weight, up: Weight, down: Weight,
                               shared: tuple[Weight, Weight, Weight] | None = None) -> int:
    sg, su, sd = shared if shared is not None else (None, None, None)
    return load_library().w4a16_moe_decode_workspace_bytes(M, top_k, xt, _dref(gate), _dref(up), _dref(down),
                                                           _dref(sg), _dref(su), _dref(sd))


def moe_decode(x: torch.Tensor, logits: torch.Tensor, top_k: int, gate: Weight, up: Weight, down: Weight,
               y: torch.Tensor, ws: torch.Tensor, shared: tuple[Weight, Weight, Weight] | None = None,
               topk_ids: torch.Tensor | None = None, topk_w: torch.Tensor | None = None, stream=None):
    """The MoE layer of a few tokens from its router logits (at most 8 float32 or 16 bfloat16 rows); y float32
    or bfloat16, shared = (gate, up, down) of a shared expert, topk_ids / topk_w receive the choice."""
    _need_x(x, gate.K)
    M = x.shape[0]
    _need(logits, "logits", torch.float32, (M, gate.num_experts))
    yt = _need_y(y, (M, down.N))
    _need(ws, "ws", torch.uint8)
    if topk_ids is not None:
        _need(topk_ids, "topk_ids", torch.int32, (M, top_k))
    if topk_w is not None:
        _need(topk_w, "topk_w", torch.float32, (M, top_k))
    sg, su, sd = shared if shared is not None else (None, None, None)
    _on_device(x=x, logits=logits, gate=gate, up=up, down=down, shared_gate=sg, shared_up=su, shared_down=sd, y=y,
               ws=ws, topk_ids=topk_ids, topk_w=topk_w)
    _check(load_library().w4a16_moe_decode(_ptr(x), _dtype_code(x), M, _ptr(logits), top_k, _dref(gate), _dref(up),
                                           _dref(down), _dref(sg), _dref(su), _dref(sd), _ptr(topk_ids), _ptr(topk_w),
                                           _ptr(y), yt, _ptr(ws), _nbytes(ws), _stream(stream)), "w4a16_moe_decode")


# ---------------------------------------------------------------- MXFP4

def mx_empty(rows: int, K: int, layout: int = MX_ROWS, device="cuda") -> MxMatrix:
    """An uninitialised MXFP4 matrix."""
    lib = load_library()
    nc, ns = lib.w4a16_mx_codes_bytes(rows, K, layout), lib.w4a16_mx_scales_bytes(rows, K, layout)
    if rows < 0 or K < 0 or (rows and K and nc == 0):
        raise ValueError(f"no MXFP4 matrix of {rows} rows of {K} in layout {layout}")
    codes = torch.empty((rows, K // 2) if layout == MX_ROWS else (nc,), dtype=torch.uint8, device=device)
    scales = torch.empty((rows, K // 32) if layout == MX_ROWS else (ns,), dtype=torch.uint8, device=device)
    return MxMatrix(codes, scales, rows, K, layout)


def _need_mx_out(out: MxMatrix, name: str, rows: int, K: int, dev: int):
    out._ready(name, dev)
    if out.rows != rows or out.K != K or out.layout != MX_ROWS:
        raise ValueError(f"{name} must be {rows} rows of {K} in ROWS, got {out.rows} of {out.K} in layout {out.layout}")


def mx_quantize(x: torch.Tensor, out: MxMatrix, stream=None):
    """x float32 or bfloat16 [rows][K] -> MXFP4 (ROWS)."""
    xt = _dtype_code(x)
    if x.dim() != 2:
        raise ValueError(f"x must be [rows][K], got {tuple(x.shape)}")
    rows, K = shape = x.shape
    dev = _device_of(x)
    _ready(x, "x", x.dtype, shape, dev)
    _need_mx_out(out, "out", rows, K, dev)
    c, s = out.codes, out.scales
    st = load_library().w4a16_mx_quantize(x.data_ptr(), xt, rows, K, c.data_ptr(), c.numel(), s.data_ptr(), s.numel(),
                                          _stream_of(stream, dev))
    if st != OK:
        raise W4A16Error(st, "w4a16_mx_quantize")


def mx_quantize_weight(w: torch.Tensor, out: MxMatrix, stream=None):
    """Weights w float32 or bfloat16 [K][N] -> MXFP4 rows of the transpose (ROWS, N rows of K)."""
    wt = _dtype_code(w)
    if w.dim() != 2:
        raise ValueError(f"w must be [K][N], got {tuple(w.shape)}")
    dev = _device_of(w)
    _ready(w, "w", w.dtype, w.shape, dev)
    _need_mx_out(out, "out", w.shape[1], w.shape[0], dev)
    _check(load_library().w4a16_mx_quantize_weight(_ptr(w), wt, w.shape[0], w.shape[1], _ptr(out.codes),
                                                   _nbytes(out.codes), _ptr(out.scales), _nbytes(out.scales),
                                                   _stream(stream)), "w4a16_mx_quantize_weight")


def mx_prepack(src: MxMatrix, dst: MxMatrix, stream=None) -> MxMatrix:
    """ROWS -> TILED, the layout the products stream, into dst's tensors; returns dst."""
    src.check("src")
    dst.check("dst")
    if (dst.rows, dst.K, dst.layout) != (src.rows, src.K, MX_TILED):
        raise ValueError(f"dst must be {src.rows} rows of {src.K} in TILED")
    out = MxDesc()
    _check(load_library().w4a16_mx_prepack(ctypes.byref(src.desc()), _ptr(dst.codes), _nbytes(dst.codes),
                                           _ptr(dst.scales), _nbytes(dst.scales), ctypes.byref(out), _stream(stream)),
           "w4a16_mx_prepack")
    return dst


def mx_dequantize(m: MxMatrix, out: torch.Tensor, stream=None):
    """The values of m [rows][K], either layout, as float32 or bfloat16."""
    ot = _dtype_code(out)
    dev = _device_of(out)
    m._ready("m", dev)
    _ready(out, "out", out.dtype, (m.rows, m.K), dev)
    st = load_library().w4a16_mx_dequantize(ctypes.byref(m.desc()), out.data_ptr(), ot, _nbytes(out),
                                            _stream_of(stream, dev))
    if st != OK:
        raise W4A16Error(st, "w4a16_mx_dequantize")


def mx_quantize_to_weight(w: torch.Tensor, stream=None) -> MxMatrix:
    """Quantize device weights [K][N] and prepack them (TILED).  With a stream, the weight is made there: the
    current one uses it once it has waited for that."""
    K, N = w.shape
    if stream is not None:
        _stream(stream)  # (of the current device)
    with torch.cuda.stream(stream):  # the rows, freed on return, are that stream's memory
        rows = mx_empty(N, K, MX_ROWS, w.device)
        mx_quantize_weight(w, rows, stream)
        out = mx_prepack(rows, mx_empty(N, K, MX_TILED, w.device), stream)
    if stream is not None:  # freed later, its memory is that stream's again when the current one is done with it
        for t in (out.codes, out.scales):
            t.record_stream(torch.cuda.current_stream())
    return out


def mx_gemm_workspace_bytes(M: int, xt: int, w: MxMatrix) -> int:
    """xt: F32, BF16, or MXFP4 for activations given as an MxMatrix."""
    lib = load_library()
    if xt == MXFP4:
        return lib.w4a16_mx_gemm_a4_workspace_bytes(M, ctypes.byref(w.desc()))
    return lib.w4a16_mx_gemm_workspace_bytes(M, xt, ctypes.byref(w.desc()))


def _mx_x(x, K: int, dev: int):
    """The type code and rows of activations [M][K]."""
    xt = _dtype_code(x)
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"activations must be [M][{K}], got {tuple(x.shape)}")
    _ready(x, "x", x.dtype, x.shape, dev)
    return xt, x.shape[0]


def _mx_io(y, M: int, N: int, ws, dev: int) -> int:
    """y float32 or bfloat16 [M][N], ws bytes; returns y's type code."""
    yt = _dtype_code(y)
    _ready(y, "y", y.dtype, (M, N), dev)
    _ready(ws, "ws", _U8, getattr(ws, "shape", None), dev)
    return yt


def mx_gemm(x, w: MxMatrix, y: torch.Tensor, ws: torch.Tensor, stream=None):
    """y = x W^T over a TILED MXFP4 weight; x a float32 or bfloat16 tensor [M][K], or an MxMatrix (ROWS)."""
    dev = _device_of(y)
    w._ready("w", dev)
    lib, d = load_library(), ctypes.byref(w.desc())
    if isinstance(x, MxMatrix):
        x._ready("x", dev)
        yt = _mx_io(y, x.rows, w.rows, ws, dev)
        st = lib.w4a16_mx_gemm_a4(ctypes.byref(x.desc()), d, y.data_ptr(), yt, ws.data_ptr(), ws.numel(),
                                  _stream_of(stream, dev))
    else:
        xt, M = _mx_x(x, w.K, dev)
        yt = _mx_io(y, M, w.rows, ws, dev)
        st = lib.w4a16_mx_gemm(x.data_ptr(), xt, M, d, y.data_ptr(), yt, ws.data_ptr(), ws.numel(),
                               _stream_of(stream, dev))
    if st != OK:
        raise W4A16Error(st, "w4a16_mx_gemm")


def mx_swiglu_mlp_workspace_bytes(M: int, xt: int, gate: MxMatrix, up: MxMatrix, down: MxMatrix) -> int:
    """xt: F32, BF16, or MXFP4 for activations given as an MxMatrix."""
    lib, d = load_library(), [ctypes.byref(w.desc()) for w in (gate, up, down)]
    if xt == MXFP4:
        return lib.w4a16_mx_swiglu_mlp_a4_workspace_bytes(M, *d)
    return lib.w4a16_mx_swiglu_mlp_workspace_bytes(M, xt, *d)


def mx_swiglu_mlp(x, gate: MxMatrix, up: MxMatrix, down: MxMatrix, y: torch.Tensor, ws: torch.Tensor, stream=None):
    """The SwiGLU MLP over TILED MXFP4 weights; x as in mx_gemm (with an MxMatrix, h is MXFP4 too)."""
    dev = _device_of(y)
    gate._ready("gate", dev), up._ready("up", dev), down._ready("down", dev)
    lib, d = load_library(), [ctypes.byref(w.desc()) for w in (gate, up, down)]
    if isinstance(x, MxMatrix):
        x._ready("x", dev)
        yt = _mx_io(y, x.rows, down.rows, ws, dev)
        st = lib.w4a16_mx_swiglu_mlp_a4(ctypes.byref(x.desc()), *d, y.data_ptr(), yt, ws.data_ptr(), ws.numel(),
                                        _stream_of(stream, dev))
    else:
        xt, M = _mx_x(x, gate.K, dev)
        yt = _mx_io(y, M, down.rows, ws, dev)
        st = lib.w4a16_mx_swiglu_mlp(x.data_ptr(), xt, M, *d, y.data_ptr(), yt, ws.data_ptr(), ws.numel(),
                                     _stream_of(stream, dev))
    if st != OK:
        raise W4A16Error(st, "w4a16_mx_swiglu_mlp")


# ---------------------------------------------------------------- norms

def block_norm(y: torch.Tensor, r: torch.Tensor | None = None, r_out: torch.Tensor | None = None, n=None, *,
               pre_w: torch.Tensor | None = None, post_w: torch.Tensor | None = None,
               gate: torch.Tensor | None = None, alpha: float = 1.0, eps: float = 1e-6, stream=None):
    """Between two blocks, one pass: r_out = r + alpha * gate * post(y), post an RMS norm with post_w (None: y);
    n = the RMS norm of r_out with pre_w.  y, r [M][H] float32 or bfloat16, r_out of r's type (y's without r; it
    may be r), n float32, bfloat16 or an MxMatrix (ROWS); post_w, pre_w [H] and gate [H] or [M][H] of one type."""
    yt = _dtype_code(y)
    if y.dim() != 2:
        raise ValueError(f"y must be [M][H], got {tuple(y.shape)}")
    M, H = shape = y.shape
    dev = _device_of(y)
    _ready(y, "y", y.dtype, shape, dev)
    residual = r if r is not None else r_out
    rt, rp, op = yt, None, None
    if residual is not None:
        rt, rd = _dtype_code(residual), residual.dtype
        if r is not None:
            _ready(r, "r", rd, shape, dev)
            rp = r.data_ptr()
        if r_out is not None:
            _ready(r_out, "r_out", rd, shape, dev)
            op = r_out.data_ptr()
    first = pre_w if pre_w is not None else post_w if post_w is not None else gate
    wt, pre, post, gp, gate_rows, row = yt, None, None, None, 1, (H,)
    if first is not None:
        wt, wd = _dtype_code(first), first.dtype
        if pre_w is not None:
            _ready(pre_w, "pre_w", wd, row, dev)
            pre = pre_w.data_ptr()
        if post_w is not None:
            _ready(post_w, "post_w", wd, row, dev)
            post = post_w.data_ptr()
        if gate is not None:
            if gate.dim() == 2:
                gate_rows = M
            _ready(gate, "gate", wd, shape if gate.dim() == 2 else row, dev)
            gp = gate.data_ptr()
    nt, np, codes, scales = F32, None, None, None
    if isinstance(n, MxMatrix):
        _need_mx_out(n, "n", M, H, dev)
        codes, scales = n.codes.data_ptr(), n.scales.data_ptr()
    elif n is not None:
        nt = _dtype_code(n)
        _ready(n, "n", n.dtype, shape, dev)
        np = n.data_ptr()
    d = NormDesc(y.data_ptr(), rp, op, post, pre, gp, gate_rows, np, codes, scales, yt, rt, wt, nt, alpha, eps)
    st = load_library().w4a16_block_norm(ctypes.byref(d), M, H, _stream_of(stream, dev))
    if st != OK:
        raise W4A16Error(st, "w4a16_block_norm")


# ---------------------------------------------------------------- helpers

def new_workspace(nbytes: int, device="cuda", stream=None) -> torch.Tensor:
    """A zero-filled workspace of at least `nbytes` bytes (16-byte aligned by torch)."""
    ws = torch.empty(max(16, (int(nbytes) + 15) // 16 * 16), dtype=torch.uint8, device=device)
    with torch.cuda.device(ws.device):
        workspace_init(ws, stream)
    return ws


def quantize_to_weight(w: torch.Tensor, stream=None) -> Weight:
    """Quantize float32 device weights [E][K][N] or [K][N] and prepack them (GROUPED).  With a stream, the weight is
    made there: the current one uses it once it has waited for that."""
    E = 1 if w.dim() == 2 else w.shape[0]
    K, N = w.shape[-2], w.shape[-1]
    if stream is not None:
        _stream(stream)  # (of the current device)
    with torch.cuda.stream(stream):  # the canonical codes, freed on return, are that stream's memory
        qw = torch.empty((E, K // 8, N), dtype=torch.int32, device=w.device)
        sc = torch.empty((E, K // GROUP, N), dtype=torch.float32, device=w.device)
        quantize(w, qw, sc, stream)
        out = prepack(Weight(qw, sc, K, N, E, LAYOUT_CANONICAL), torch.empty_like(qw), stream)
    if stream is not None:  # freed later, its memory is that stream's again when the current one is done with it
        for t in (out.qw, out.scales):
            t.record_stream(torch.cuda.current_stream())
    return out
