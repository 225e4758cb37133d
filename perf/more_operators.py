"""Workloads of the MXFP4 operators (quantisation, products, SwiGLU MLP) and of the
norms round a block.

Each case is one call of an operator on data a serving engine has in hand: weights in
MXFP4 (E2M1 codes, one E8M0 scale per 32 values along K), activations, norm weights.
``run`` computes it in elementary torch operations, or with ``own`` through the
library.  Sizes are the synthetic shapes of ``workloads.CONFIGS`` (hidden 7168, dense
intermediate 18432, one tensor-parallel share of it 2304, GEMM 256 x 512 and
7168 x 4096, 1733 rows of the busiest expert) and odd ones.
"""
from __future__ import annotations

import math

import torch

own = False

# ---------------------------------------------------------------- cases


def _named(c, name):
    return dict(c, name=name) if name else c


def _quantize(name, M, K, xt):
    return _named(dict(op="quantize", M=M, K=K, xt=xt), name)


def _gemm(name, M, K, N, xt, yt):
    """``xt`` "mx": the activations are MXFP4 rows too."""
    return _named(dict(op="gemm", M=M, K=K, N=N, xt=xt, yt=yt), name)


def _mlp(name, M, H, I, xt, yt):
    return _named(dict(op="mlp", M=M, H=H, I=I, xt=xt, yt=yt), name)


def _norm(name, M, H, t, nt, post=True, gate="channel", alpha=1.0):
    """``t``: type of the block's output and the residual stream, ``nt`` of the normed
    rows ("mx": MXFP4); ``gate``: "none", "channel" [H] or "row" [M][H]."""
    return _named(dict(op="norm", M=M, H=H, t=t, nt=nt, post=post, gate=gate, alpha=alpha), name)


def listed():
    return [
        # one token's activations to MXFP4: pure latency
        _quantize("mx_quantize_m1_bf16", 1, 7168, "bf16"),
        # a prompt's rows, an odd number of them
        _quantize("mx_quantize_m1733_f32", 1733, 7168, "f32"),
        # one token through the smallest GEMM of the configurations: latency
        _gemm("mx_gemm_m1_small_f32", 1, 256, 512, "f32", "f32"),
        # sixteen decoding requests
        _gemm("mx_gemm_m16_bf16", 16, 7168, 4096, "bf16", "bf16"),
        # an odd batch over one share of a tensor-parallel down projection
        _gemm("mx_gemm_m37_f32", 37, 2304, 7168, "f32", "f32"),
        # a prompt through the configurations' large GEMM, 16-bit activations
        _gemm("mx_gemm_m2048_bf16", 2048, 7168, 4096, "bf16", "bf16"),
        # the same with 4-bit activations
        _gemm("mx_gemm_a4_m2048", 2048, 7168, 4096, "mx", "bf16"),
        # four decoding requests through the dense MLP
        _mlp("mx_mlp_m4_f32", 4, 7168, 18432, "f32", "f32"),
        # a verify batch through the dense MLP
        _mlp("mx_mlp_m64_bf16", 64, 7168, 18432, "bf16", "bf16"),
        # a prompt through the dense MLP, 4-bit activations
        _mlp("mx_mlp_a4_m1024", 1024, 7168, 18432, "mx", "bf16"),
        # four decoding requests: post-norm, gate, residual, next pre-norm
        _norm("block_norm_m4_bf16", 4, 7168, "bf16", "bf16"),
        # a prompt's rows, the next block's activations straight to MXFP4
        _norm("block_norm_m2048_mx", 2048, 7168, "bf16", "mx", gate="row", alpha=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm", "mlp", "mlp", "norm"))
    if op == "quantize":
        return _quantize(None, _log(rng, 1, 2048), _mult(rng, 32, 7168, 32), rng.choice(("f32", "bf16")))
    if op == "norm":
        t = rng.choice(("f32", "bf16"))
        return _norm(None, _log(rng, 1, 2048), _mult(rng, 64, 7168, 32), t, rng.choice((t, "mx")),
                     rng.random() < 0.6, rng.choice(("none", "channel", "row")), rng.choice((1.0, 0.5, 0.25)))
    xt = rng.choice(("f32", "bf16", "mx"))
    yt = "f32" if xt == "f32" else "bf16"
    if op == "gemm":
        return _gemm(None, _log(rng, 1, 2048), _mult(rng, 128, 7168, 32), _mult(rng, 128, 7168, 16), xt, yt)
    return _mlp(None, _log(rng, 1, 1024), _mult(rng, 256, 7168, 32), _mult(rng, 256, 18432, 32), xt, yt)


# ---------------------------------------------------------------- the format

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # E2M1 codes 0 to 7; 8 to 15 are their negatives


def _quantized(x):
    """Codes (0 to 15) and scale bytes of x's blocks of 32 along the last axis: the scale is
    2^(floor(log2 max|x|) - 2), a code the nearest value, ties to the even code, at most 6."""
    b = x.unflatten(-1, (-1, 32))
    _, e = torch.frexp(b.abs().amax(-1))  # max|x| = m 2^e, m in [1/2, 1)
    s = torch.where(b.abs().amax(-1) > 0, (e - 3).clamp(min=-127), torch.full_like(e, -127))
    v = torch.ldexp(b.double(), -s.unsqueeze(-1)).abs()
    # one step per border between neighbouring codes; a border itself goes to the even code
    q = (v > 0.25).int() + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5)
    q = q + 8 * torch.signbit(b)
    return q.flatten(-2).to(torch.uint8), (s + 127).to(torch.uint8)


def _packed(q):
    return q[..., 0::2] | q[..., 1::2] << 4  # the lower k in the low half


def _values(codes, scales):
    """float32 values [rows][K] of codes [rows][K/2] and scales [rows][K/32]."""
    table = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=codes.device)
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = table[q.int()].unflatten(-1, (-1, 32))
    return torch.ldexp(v, (scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _tiled(codes, scales):
    """The TILED layout the products stream: rows padded to 64 and K to 128 with zeros."""
    n, kb = codes.shape
    J, S = -(-n // 64), -(-kb // 64)
    c = torch.zeros((J * 64, S * 64), dtype=torch.uint8, device=codes.device)
    c[:n, :kb] = codes
    s = torch.full((J * 64, S * 4), 127, dtype=torch.uint8, device=codes.device)
    s[:n, :scales.shape[1]] = scales
    c = c.view(J, 4, 16, S, 4, 16).permute(0, 3, 1, 4, 2, 5).contiguous()  # 64 rows, step, 16 rows, k block, row, byte
    s = s.view(J, 4, 16, S, 4).permute(0, 3, 4, 2, 1).contiguous()  # 64 rows, step, k block, row, 16 rows
    return c, s


# ---------------------------------------------------------------- inputs


def _act(g, M, K, xt):
    x = torch.randn((M, K), generator=g, device="cuda")
    return x.to(torch.bfloat16) if xt == "bf16" else x


def _weight(g, K, N):
    """An MXFP4 weight [N][K] of standard deviation 0.02, as saved and as the library streams it."""
    q, s = _quantized(torch.randn((N, K), generator=g, device="cuda") * 0.02)
    c = _packed(q)
    return {"codes": c, "scales": s, "tiled": _tiled(c, s), "K": K, "N": N}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    M = c["M"]
    if c["op"] == "quantize":
        s["x"] = _act(g, M, c["K"], c["xt"])
        return s
    if c["op"] == "norm":
        H, t = c["H"], _TYPES[c["t"]]
        s["y"] = (torch.randn((M, H), generator=g, device="cuda") * 0.7).to(t)
        s["r"] = (torch.randn((M, H), generator=g, device="cuda") * 3).to(t)
        s["pre"] = (1 + torch.randn((H,), generator=g, device="cuda") * 0.1).to(t)
        s["post"] = (1 + torch.randn((H,), generator=g, device="cuda") * 0.1).to(t) if c["post"] else None
        shape = {"none": None, "channel": (H,), "row": (M, H)}[c["gate"]]
        s["gate"] = None if shape is None else torch.randn(shape, generator=g, device="cuda").to(t)
        return s
    if c["op"] == "gemm":
        shapes = [(c["K"], c["N"])]
    else:
        shapes = [(c["H"], c["I"]), (c["H"], c["I"]), (c["I"], c["H"])]
    s["w"] = [_weight(g, K, N) for K, N in shapes]
    s["x"] = _act(g, M, shapes[0][0], c["xt"])
    if c["xt"] == "mx":
        q, sc = _quantized(s.pop("x"))
        s["xq"] = (_packed(q), sc)
    return s


# ---------------------------------------------------------------- plain forms

EPS = 1e-6


def _silu(z):
    return z / (1 + torch.exp(-z))


def _rms(v, w):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w


def _plain_norm(s):
    c = s["case"]
    wide = torch.float64 if c["nt"] == "mx" else torch.float32  # codes have borders: 64 bits
    y, r = s["y"].to(wide), s["r"].to(wide)
    if c["post"]:
        y = _rms(y, s["post"].to(wide))
    if s["gate"] is not None:
        y = y * s["gate"].to(wide)
    r = (r + c["alpha"] * y).to(s["r"].dtype)
    n = _rms(r.to(wide), s["pre"].to(wide))
    if c["nt"] != "mx":
        return {"r": r, "n": n.to(_TYPES[c["nt"]])}
    q, sc = _quantized(n)
    return {"r": r, "n": _values(_packed(q), sc).to(torch.bfloat16)}


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _plain_norm(s)
    if c["op"] == "quantize":
        q, sc = _quantized(s["x"])
        return {"values": _values(_packed(q), sc).to(s["x"].dtype), "scales": sc}
    x = _values(*s["xq"]) if c["xt"] == "mx" else s["x"].float()
    w = [_values(w["codes"], w["scales"]) for w in s["w"]]
    if c["op"] == "gemm":
        return (x @ w[0].t()).to(_TYPES[c["yt"]])
    h = _silu(x @ w[0].t()) * (x @ w[1].t())
    if c["xt"] == "mx":
        q, sc = _quantized(h)
        h = _values(_packed(q), sc)
    return (h @ w[2].t()).to(_TYPES[c["yt"]])


# ---------------------------------------------------------------- the library's calls


def _handles(s):
    """What a serving program keeps: descriptors, a workspace and output buffers."""
    import int4_w4a16_group_g32_amd as L

    c, M = s["case"], s["case"]["M"]
    o = {"L": L}

    def rows(K):
        return L.MxMatrix(torch.empty((M, K // 2), dtype=torch.uint8, device="cuda"),
                          torch.empty((M, K // 32), dtype=torch.uint8, device="cuda"), M, K, L.MX_ROWS)

    if c["op"] == "quantize":
        o["m"] = rows(c["K"])
        o["values"] = torch.empty_like(s["x"])
        return o
    if c["op"] == "norm":
        o["r"] = torch.empty_like(s["r"])
        o["n"] = rows(c["H"]) if c["nt"] == "mx" else torch.empty_like(s["r"])
        o["values"] = torch.empty((M, c["H"]), dtype=torch.bfloat16, device="cuda") if c["nt"] == "mx" else None
        return o
    o["w"] = [L.MxMatrix(*w["tiled"], w["N"], w["K"], L.MX_TILED) for w in s["w"]]
    if c["xt"] == "mx":
        o["x"] = L.MxMatrix(*s["xq"], M, o["w"][0].K, L.MX_ROWS)
        xt = L.MXFP4
    else:
        o["x"] = s["x"]
        xt = L.BF16 if c["xt"] == "bf16" else L.F32
    o["y"] = torch.empty((M, o["w"][-1].rows), dtype=_TYPES[c["yt"]], device="cuda")
    size = L.mx_gemm_workspace_bytes if c["op"] == "gemm" else L.mx_swiglu_mlp_workspace_bytes
    o["ws"] = L.new_workspace(size(M, xt, *o["w"]))
    return o


def _own(s):
    c = s["case"]
    o = s.get("handles")
    if o is None:
        o = s["handles"] = _handles(s)
    L = o["L"]
    if c["op"] == "quantize":
        L.mx_quantize(s["x"], o["m"])
        L.mx_dequantize(o["m"], o["values"])
        return {"values": o["values"], "scales": o["m"].scales}
    if c["op"] == "norm":
        L.block_norm(s["y"], s["r"], o["r"], o["n"], pre_w=s["pre"], post_w=s["post"], gate=s["gate"],
                     alpha=c["alpha"], eps=EPS)
        if c["nt"] == "mx":
            L.mx_dequantize(o["n"], o["values"])
            return {"r": o["r"], "n": o["values"]}
        return {"r": o["r"], "n": o["n"]}
    if c["op"] == "gemm":
        L.mx_gemm(o["x"], o["w"][0], o["y"], o["ws"])
    else:
        L.mx_swiglu_mlp(o["x"], *o["w"], o["y"], o["ws"])
    return o["y"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work and exact values

_BYTES = {"f32": 4, "bf16": 2, "mx": 17 / 32}


def work(case):
    c = case
    M = c["M"]
    if c["op"] == "quantize":  # the rows, their codes and scales, and the values these stand for
        return {"bytes": M * c["K"] * (2 * _BYTES[c["xt"]] + 17 / 32), "flops": 4 * M * c["K"]}
    if c["op"] == "norm":
        H, b = c["H"], _BYTES[c["t"]]
        gate = {"none": 0, "channel": H, "row": M * H}[c["gate"]]
        out = 2 + 17 / 32 if c["nt"] == "mx" else _BYTES[c["nt"]]
        return {"bytes": M * H * (3 * b + out) + b * (gate + H * (1 + bool(c["post"]))), "flops": 10 * M * H}
    if c["op"] == "gemm":
        weights, inout = c["K"] * c["N"], (c["K"], c["N"])
    else:
        weights, inout = 3 * c["H"] * c["I"], (c["H"], c["H"])
    return {"bytes": weights * 17 / 32 + M * (inout[0] * _BYTES[c["xt"]] + inout[1] * _BYTES[c["yt"]]),
            "flops": 2 * M * weights}


def _exact_values(codes, scales):
    """64-bit values of codes and scales, from the bits of the codes: sign, two of exponent, one of mantissa."""
    out = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.float64, device=codes.device)
    for half in range(2):
        q = (codes // 16 if half else codes % 16).long()
        e, m = q // 2 % 4, (q % 2).double()
        mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, (e - 1).double()))
        out[:, half::2] = torch.where(q >= 8, -mag, mag)
    return out * torch.pow(2.0, scales.double() - 127).repeat_interleave(32, 1)


def _exact_round(x):
    """x (64 bits) rounded to MXFP4, as values: the nearest multiple of each binade's step."""
    b = x.reshape(x.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(torch.where(top > 0, top, 1.0))), -125.0)
    e = torch.where(torch.pow(2.0, e) > top, e - 1, e)
    e = torch.where(torch.pow(2.0, e + 1) <= top, e + 1, e)
    s = torch.pow(2.0, torch.clamp(e - 2, min=-127.0))
    v = b / s
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    v = torch.clamp(torch.round(v / step) * step, -6, 6)  # halfway cases to the even multiple, which is the even code
    return (v * s).reshape(x.shape), (torch.clamp(e - 2, min=-127.0) + 127).reshape(x.shape[0], -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantize":
        v, sc = _exact_round(s["x"].double())
        return {"values": v, "scales": sc.to(torch.uint8)}
    if c["op"] == "norm":
        y, r = s["y"].double(), s["r"].double()
        if c["post"]:
            y = y * torch.rsqrt(y.square().sum(1, keepdim=True) / c["H"] + EPS) * s["post"].double()
        if s["gate"] is not None:
            y = s["gate"].double() * y
        r = r + y * c["alpha"]
        n = r.to(s["r"].dtype).double()  # the residual stream is stored in its own type
        n = n * torch.rsqrt(n.square().sum(1, keepdim=True) / c["H"] + EPS) * s["pre"].double()
        return {"r": r, "n": _exact_round(n)[0] if c["nt"] == "mx" else n}
    x = _exact_values(*s["xq"]) if c["xt"] == "mx" else s["x"].double()
    w = [_exact_values(w["codes"], w["scales"]) for w in s["w"]]
    if c["op"] == "gemm":
        return torch.matmul(w[0], x.t()).t().contiguous()
    g, u = torch.matmul(x, w[0].t()), torch.matmul(x, w[1].t())
    h = g * torch.sigmoid(g) * u
    if c["xt"] == "mx":
        h = _exact_round(h)[0]
    return torch.matmul(h, w[2].t())
