"""Workloads of the low-rank-adapter projections and the few-token MoE layer.

Each case is one call of an operator on data a serving engine has in hand: W4A16
weights in the GROUPED layout, adapters as they are trained and saved, activations,
router logits.  ``run`` computes it in elementary torch operations, or with ``own``
through the library.  Sizes are the synthetic shapes of ``workloads.CONFIGS``
(hidden 7168, dense intermediate 18432, one tensor-parallel share of it 2304, expert
intermediate 2048, 384 experts, top-8, GEMM 256 x 512 and 7168 x 4096) and odd ones.
"""
from __future__ import annotations

import math

import torch

own = False

# ---------------------------------------------------------------- cases


def _gemm(name, M, K, N, R, n, xt, mix="rows", gs=32, ranked=False):
    """``n`` adapters of rank ``R``; mix "rows": every row has an adapter of its own
    choosing (one decoding request a row), "segments": runs of rows share one
    (prompts of several requests); ``ranked``: the adapters' ranks differ."""
    c = dict(op="gemm", M=M, K=K, N=N, R=R, n=n, xt=xt, mix=mix, gs=gs, ranked=ranked)
    return dict(c, name=name) if name else c


def _mlp(name, M, H, I, R, n, xt, mix="rows", gs=32, ranked=False):
    c = dict(op="mlp", M=M, H=H, I=I, R=R, n=n, xt=xt, mix=mix, gs=gs, ranked=ranked)
    return dict(c, name=name) if name else c


def _moe(name, M, H, I, E, k, xt, shared=False, gs=32):
    c = dict(op="moe", M=M, H=H, I=I, E=E, k=k, xt=xt, shared=shared, gs=gs)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through the smallest GEMM of the configurations: pure latency
        _gemm("lora_gemm_m1_small_f32", 1, 256, 512, 8, 4, "f32"),
        # sixteen decoding requests, nearly every one with its own adapter
        _gemm("lora_gemm_m16_bf16", 16, 7168, 4096, 16, 32, "bf16"),
        # an odd batch over one share of a tensor-parallel down projection, ranks that differ
        _gemm("lora_gemm_m37_f32", 37, 2304, 7168, 40, 8, "f32", ranked=True),
        # a full verify batch over many tenants, scale groups of 64
        _gemm("lora_gemm_m64_bf16", 64, 7168, 4096, 32, 64, "bf16", gs=64),
        # prompts of a few requests, the configurations' large GEMM
        _gemm("lora_gemm_m2048_bf16", 2048, 7168, 4096, 64, 8, "bf16", mix="segments"),
        # four decoding requests through the dense MLP
        _mlp("lora_mlp_m4_f32", 4, 7168, 18432, 16, 8, "f32"),
        # a verify batch through the dense MLP
        _mlp("lora_mlp_m64_bf16", 64, 7168, 18432, 16, 16, "bf16"),
        # three tokens through a small layer: latency
        _moe("moe_m3_small_f32", 3, 256, 128, 6, 2, "f32"),
        # one token through the routed layer: what a single stream waits for
        _moe("moe_m1_bf16", 1, 7168, 2048, 384, 8, "bf16"),
        # four tokens of a short draft, float32 activations
        _moe("moe_m4_f32", 4, 7168, 2048, 384, 8, "f32"),
        # sixteen tokens with the shared expert: the most this form takes
        _moe("moe_m16_shared_bf16", 16, 7168, 2048, 384, 8, "bf16", shared=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log(rng, lo, hi) // m * m)


def draw(rng):
    xt = rng.choice(("f32", "bf16"))
    gs = rng.choice((32, 32, 64, 128))
    op = rng.choice(("gemm", "gemm", "mlp", "moe", "moe"))
    if op == "moe":
        M = rng.randint(1, 8 if xt == "f32" else 16)
        E = _log(rng, 4, 384)
        k = rng.randint(1, min(8, E))
        return _moe(None, M, _mult(rng, 256, 7168, 128), _mult(rng, 128, 2048, 128), E, k, xt,
                    rng.random() < 0.4, gs)
    R = 8 * rng.choice((1, 2, 2, 3, 4, 5, 8))
    n = _log(rng, 1, 64)
    mix = rng.choice(("rows", "segments"))
    ranked = rng.random() < 0.4
    if op == "gemm":
        return _gemm(None, _log(rng, 1, 1500), _mult(rng, 256, 7168, 128), _mult(rng, 256, 4096, 64), R, n, xt, mix,
                     gs, ranked)
    return _mlp(None, _log(rng, 1, 200), _mult(rng, 256, 4096, 128), _mult(rng, 256, 8192, 128), R, n, xt, mix, gs,
                ranked)


# ---------------------------------------------------------------- inputs


def _weight(g, K, N, gs, E=1):
    """Random code words (every nibble equally likely) in the GROUPED layout and
    float32 scales as max|w| / 7 gives them for weights of standard deviation 0.02."""
    qw = torch.randint(-(2 ** 31), 2 ** 31, (E, K // 32, N // 64, 64, 4), generator=g, device="cuda",
                       dtype=torch.int32)
    sc = torch.rand((E, K // gs, N), generator=g, device="cuda") * 0.005 + 0.004
    return {"qw": qw, "sc": sc, "K": K, "N": N, "gs": gs, "E": E}


def _act(g, M, K, xt):
    x = torch.randn((M, K), generator=g, device="cuda")
    return x.to(torch.bfloat16) if xt == "bf16" else x


def _adapters(g, n, R, K, N, ranks):
    """A [n][R][K] and B [n][N][R] in bf16, one scale each (alpha / rank)."""
    a = (torch.randn((n, R, K), generator=g, device="cuda") / math.sqrt(K)).to(torch.bfloat16)
    b = (torch.randn((n, N, R), generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    s = torch.rand((n,), generator=g, device="cuda") + 0.5
    return {"a": a, "b": b, "s": s, "ranks": ranks}


def _adapter_ids(g, M, n, mix):
    """One id a row in [0, n), or -1 for one request in eight (no adapter)."""
    if mix == "rows":
        of_row = torch.arange(M, device="cuda")
    else:  # about one request per 128 rows, borders anywhere
        border = torch.rand((M,), generator=g, device="cuda") < 1 / 128
        of_row = torch.cumsum(border.to(torch.int64), 0)
    ids = torch.randint(0, n, (M,), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.rand((M,), generator=g, device="cuda") < 0.125] = -1
    return ids[of_row].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] == "moe":
        H, I, E, gs = c["H"], c["I"], c["E"], c["gs"]
        s["w"] = [_weight(g, H, I, gs, E), _weight(g, H, I, gs, E), _weight(g, I, H, gs, E)]
        if c["shared"]:
            s["ws"] = [_weight(g, H, I, gs), _weight(g, H, I, gs), _weight(g, I, H, gs)]
        s["x"] = _act(g, c["M"], H, c["xt"])
        s["logits"] = torch.randn((c["M"], E), generator=g, device="cuda")
        return s
    n, R = c["n"], c["R"]
    ranks = None
    if c["ranked"]:
        ranks = torch.randint(1, R + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    if c["op"] == "gemm":
        shapes = [(c["K"], c["N"])]
    else:
        shapes = [(c["H"], c["I"]), (c["H"], c["I"]), (c["I"], c["H"])]
    s["w"] = [_weight(g, K, N, c["gs"]) for K, N in shapes]
    s["lora"] = [_adapters(g, n, R, K, N, ranks) for K, N in shapes]
    s["ids"] = _adapter_ids(g, c["M"], n, c["mix"])
    s["x"] = _act(g, c["M"], shapes[0][0], c["xt"])
    return s


# ---------------------------------------------------------------- plain forms


def _dequant(w, experts=None):
    """float32 weights [E][K][N] of GROUPED codes (of the listed experts)."""
    qw = w["qw"] if experts is None else w["qw"][experts]
    sc = w["sc"] if experts is None else w["sc"][experts]
    shifts = torch.arange(0, 32, 4, device=qw.device, dtype=torch.int32)
    E, G, J = qw.shape[:3]
    q = ((qw.view(E, G, J, 4, 16, 4, 1) >> shifts) & 15) - 8  # e, g, j, b, l, c, i
    q = q.permute(0, 1, 3, 6, 2, 4, 5).reshape(E, w["K"], w["N"]).to(torch.float32)
    q.view(E, -1, w["gs"], w["N"]).mul_(sc.unsqueeze(2))
    return q


def _lora_term(x, lo, ids):
    """s_a (x A_a^T) B_a^T with each row's adapter a; rows without one are zero."""
    a, b = lo["a"].float(), lo["b"].float()
    n, R, _ = a.shape
    t = (x @ a.view(n * R, -1).t()).view(-1, n, R)  # every adapter's product, then each row's own
    use = torch.arange(n, device=x.device) == ids.unsqueeze(1)
    t = t * (use * lo["s"]).unsqueeze(2)
    if lo["ranks"] is not None:
        t = t * (torch.arange(R, device=x.device) < lo["ranks"].unsqueeze(1))
    return t.view(-1, n * R) @ b.permute(0, 2, 1).reshape(n * R, -1)


def _silu(z):
    return z / (1 + torch.exp(-z))


def _plain(s):
    c, x = s["case"], s["x"].float()
    out = torch.bfloat16 if c["xt"] == "bf16" else torch.float32
    if c["op"] == "gemm":
        return (x @ _dequant(s["w"][0])[0] + _lora_term(x, s["lora"][0], s["ids"])).to(out)
    if c["op"] == "mlp":
        g = x @ _dequant(s["w"][0])[0] + _lora_term(x, s["lora"][0], s["ids"])
        u = x @ _dequant(s["w"][1])[0] + _lora_term(x, s["lora"][1], s["ids"])
        h = _silu(g) * u
        return (h @ _dequant(s["w"][2])[0] + _lora_term(h, s["lora"][2], s["ids"])).to(out)
    val, idx = torch.sort(s["logits"], dim=1, descending=True, stable=True)  # ties: lowest index first
    val, idx = val[:, :c["k"]], idx[:, :c["k"]]
    p = torch.exp(val - val[:, :1])
    p = p / p.sum(1, keepdim=True)
    e = idx.reshape(-1)
    xp = x.repeat_interleave(c["k"], 0).unsqueeze(1)  # one row a (token, expert) pair
    h = _silu(torch.bmm(xp, _dequant(s["w"][0], e))) * torch.bmm(xp, _dequant(s["w"][1], e))
    o = torch.bmm(h, _dequant(s["w"][2], e)).view(c["M"], c["k"], -1)
    y = (p.unsqueeze(2) * o).sum(1)
    if c["shared"]:
        g, u, d = (_dequant(w)[0] for w in s["ws"])
        y = y + (_silu(x @ g) * (x @ u)) @ d
    return {"y": y.to(out), "ids": idx.to(torch.int32), "weights": p}


# ---------------------------------------------------------------- the library's calls


def _handles(s):
    """What a serving program keeps: descriptors of its weights and adapters, a
    workspace and output buffers."""
    import int4_w4a16_group_g32_amd as L

    c = s["case"]

    def weight(w):
        return L.Weight(w["qw"], w["sc"], w["K"], w["N"], w["E"], L.LAYOUT_GROUPED, w["gs"])

    xt = L.BF16 if c["xt"] == "bf16" else L.F32
    o = {"L": L, "w": [weight(w) for w in s["w"]]}
    N = c["N"] if c["op"] == "gemm" else c["H"]
    o["y"] = torch.empty((c["M"], N), dtype=s["x"].dtype, device="cuda")
    if c["op"] == "moe":
        o["shared"] = tuple(weight(w) for w in s["ws"]) if c["shared"] else None
        o["ids"] = torch.empty((c["M"], c["k"]), dtype=torch.int32, device="cuda")
        o["p"] = torch.empty((c["M"], c["k"]), dtype=torch.float32, device="cuda")
        nbytes = L.moe_decode_workspace_bytes(c["M"], c["k"], xt, *o["w"], shared=o["shared"])
    else:
        o["lora"] = [L.Lora(a["a"], a["b"], a["s"], a["ranks"]) for a in s["lora"]]
        if c["op"] == "gemm":
            nbytes = L.gemm_lora_workspace_bytes(c["M"], o["w"][0], xt, o["lora"][0])
        else:
            nbytes = L.swiglu_mlp_lora_workspace_bytes(c["M"], xt, *o["w"], *o["lora"])
    o["ws"] = L.new_workspace(nbytes)
    return o


def _own(s):
    c = s["case"]
    o = s.get("handles")
    if o is None:
        o = s["handles"] = _handles(s)
    L = o["L"]
    if c["op"] == "gemm":
        L.gemm_lora(s["x"], o["w"][0], o["lora"][0], s["ids"], o["y"], o["ws"])
        return o["y"]
    if c["op"] == "mlp":
        L.swiglu_mlp_lora(s["x"], *o["w"], *o["lora"], s["ids"], o["y"], o["ws"])
        return o["y"]
    L.moe_decode(s["x"], s["logits"], c["k"], *o["w"], o["y"], o["ws"], shared=o["shared"], topk_ids=o["ids"],
                 topk_w=o["p"])
    return {"y": o["y"], "ids": o["ids"], "weights": o["p"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work and exact values


def work(case):
    c = case
    xb = 2 if c["xt"] == "bf16" else 4
    per = 0.5 + 4 / c["gs"]  # bytes of one weight
    M = c["M"]
    if c["op"] == "moe":
        H, I, E, k = c["H"], c["I"], c["E"], c["k"]
        distinct = E * (1 - (1 - k / E) ** M)  # experts that occur, on average
        experts, rows = distinct + bool(c["shared"]), M * (k + bool(c["shared"]))
        return {"bytes": experts * 3 * H * I * per + 2 * M * H * xb + 4 * M * E + 8 * M * k,
                "flops": rows * 6 * H * I}
    n, R = c["n"], c["R"]
    requests = M if c["mix"] == "rows" else 1 + (M - 1) / 128
    used = n * (1 - (1 - 0.875 / n) ** requests)  # adapters that occur, on average
    rank = (R + 1) / 2 if c["ranked"] else R
    if c["op"] == "gemm":
        shapes, inout = [(c["K"], c["N"])], c["K"] + c["N"]
    else:
        shapes, inout = [(c["H"], c["I"]), (c["H"], c["I"]), (c["I"], c["H"])], 2 * c["H"]
    return {"bytes": sum(K * N * per + used * 2 * rank * (K + N) for K, N in shapes) + M * inout * xb + 4 * M,
            "flops": sum(2 * M * (K * N + 0.875 * rank * (K + N)) for K, N in shapes)}


def _exact_weight(w, e):
    """Expert e's weights [K][N] in 64 bits, from the bytes of its code words."""
    K, N = w["K"], w["N"]
    by = w["qw"][e].view(torch.uint8).view(K // 32, N // 64, 4, 16, 4, 4)  # block, columns / 64, word, slot, column, byte
    out = torch.empty((K // 32, 4, 4, 2, N // 64, 16, 4), dtype=torch.float64, device=by.device)
    for i in range(4):  # byte i: row 2i in its low half, row 2i + 1 in its high half
        out[:, :, i, 0] = (by[..., i] % 16).double().transpose(1, 2) - 8
        out[:, :, i, 1] = (by[..., i] // 16).double().transpose(1, 2) - 8
    return out.reshape(K, N) * w["sc"][e].double().repeat_interleave(w["gs"], 0)


def _exact_linear(x, w, lo, ids):
    y = x @ _exact_weight(w, 0)
    for a in sorted(set(ids.tolist()) - {-1}):
        r = lo["a"].shape[1] if lo["ranks"] is None else int(lo["ranks"][a])
        rows = (ids == a).nonzero().view(-1)
        t = x[rows] @ lo["a"][a, :r].double().t()
        y[rows] += lo["s"][a].double() * (t @ lo["b"][a, :, :r].double().t())
    return y


def _exact_glu(g, u):
    return g * torch.sigmoid(g) * u


def exact(case, seed):
    s = prepare(case, seed)
    c, x = s["case"], s["x"].double()
    if c["op"] == "gemm":
        return _exact_linear(x, s["w"][0], s["lora"][0], s["ids"])
    if c["op"] == "mlp":
        h = _exact_glu(*(_exact_linear(x, s["w"][i], s["lora"][i], s["ids"]) for i in (0, 1)))
        return _exact_linear(h, s["w"][2], s["lora"][2], s["ids"])
    logits = s["logits"].double().cpu()
    ids = torch.tensor([sorted(range(c["E"]), key=lambda e: (-row[e], e))[:c["k"]] for row in logits.tolist()])
    p = torch.softmax(torch.gather(logits, 1, ids), 1).cuda()
    y = torch.zeros_like(x)
    for e in sorted(set(ids.view(-1).tolist())):
        rows, slot = (ids == e).nonzero(as_tuple=True)
        rows, slot = rows.cuda(), slot.cuda()
        h = _exact_glu(x[rows] @ _exact_weight(s["w"][0], e), x[rows] @ _exact_weight(s["w"][1], e))
        y[rows] += p[rows, slot].unsqueeze(1) * (h @ _exact_weight(s["w"][2], e))
    if c["shared"]:
        g, u, d = (_exact_weight(w, 0) for w in s["ws"])
        y += _exact_glu(x @ g, x @ u) @ d
    return {"y": y, "ids": ids.to(torch.int32).cuda(), "weights": p}
