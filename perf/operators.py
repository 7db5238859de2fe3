"""The dense feed-forward operators beside the MoE layer: cases, inputs, plain forms and exact values.

Five kinds of case:
  ffn       gated feed-forward block, forward: y = (silu(x Wg^T) * (x Wu^T)) Wd^T, with or without the saved g and u
  ffn_grad  its backward pass from the saved g and u: dx, dWg, dWu, dWd
  product   matrix product of int8 codes with a scale per token and per output channel
  linear    the same from 16-bit tokens: quantise the tokens, then the product
  int_ffn   the gated block on int8 weights, from 16-bit tokens to 16-bit outputs

Weights are [out][in] row-major.  Quantisation of a row: scale = fp32(max|row| / 127), code = row / scale rounded
to the nearest integer, ties to even (a row of zeros has scale 0 and codes 0).
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one token through a small dense block (the Qwen-A3B-shaped expert's sizes): latency
        {"name": "ffn one token", "kind": "ffn", "T": 1, "H": 2048, "I": 768, "type": "bf16", "save": False, "pad": 0},
        # a decode batch through an always-on block of the GLM-shaped layer: weight bandwidth
        {"name": "ffn decode batch", "kind": "ffn", "T": 32, "H": 6144, "I": 2048, "type": "bf16", "save": False, "pad": 0},
        # a ragged prompt, tokens taken as a slice of a wider buffer
        {"name": "ffn ragged prompt", "kind": "ffn", "T": 1531, "H": 7168, "I": 2048, "type": "fp16", "save": False, "pad": 64},
        # forward pass of a training step, g and u kept for the backward pass
        {"name": "ffn training forward", "kind": "ffn", "T": 8192, "H": 7168, "I": 2048, "type": "bf16", "save": True, "pad": 0},
        # gradients of a few rows (short fine-tuning samples): weights dominate
        {"name": "ffn gradient, few rows", "kind": "ffn_grad", "T": 77, "H": 2048, "I": 768, "type": "bf16", "pad": 0},
        # gradients of an ordinary batch of a small block
        {"name": "ffn gradient", "kind": "ffn_grad", "T": 4096, "H": 2048, "I": 768, "type": "fp16", "pad": 0},
        # gradients of a large batch of the DeepSeek-shaped block: matrix rate
        {"name": "ffn gradient, large", "kind": "ffn_grad", "T": 8192, "H": 7168, "I": 2048, "type": "bf16", "pad": 0},
        # one token's projection with codes in hand (several projections share them)
        {"name": "product one token", "kind": "product", "T": 1, "K": 7168, "N": 4096, "type": "bf16", "pad": 0},
        # a prefill chunk's projection with codes in hand
        {"name": "product prefill", "kind": "product", "T": 4096, "K": 6144, "N": 6144, "type": "bf16", "pad": 0},
        # a ragged chunk into an odd number of channels, 32-bit results
        {"name": "linear ragged", "kind": "linear", "T": 1021, "K": 2048, "N": 5003, "type": "bf16", "out": "fp32", "pad": 0},
        # a small decode batch through the int8 block
        {"name": "int8 ffn decode batch", "kind": "int_ffn", "T": 16, "H": 7168, "I": 2048, "type": "bf16", "pad": 0},
        # a full prefill chunk through the int8 block
        {"name": "int8 ffn prefill", "kind": "int_ffn", "T": 8192, "H": 7168, "I": 2048, "type": "bf16", "pad": 0},
    ]


def _width(rng, lo, hi):
    """A width of a model: mostly multiples of 64, some of 16, now and then any number."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    step = rng.choice([64, 64, 64, 64, 64, 64, 16, 16, 16, 1])
    return max(1, int(round(v / step)) * step)


def draw(rng):
    kind = rng.choice(["ffn", "ffn", "ffn_grad", "ffn_grad", "product", "linear", "int_ffn"])
    # lengths of one token to 8192, over their logarithm
    T = int(math.exp(rng.uniform(0.0, math.log(8192.0))))
    c = {"kind": kind, "T": max(1, T), "type": rng.choice(["bf16", "bf16", "fp16"]), "pad": rng.choice([0, 0, 64])}
    if kind in ("product", "linear"):
        c["K"], c["N"] = _width(rng, 256, 7168), _width(rng, 256, 7168)
        c["type"] = rng.choice(["bf16", "fp16", "fp32"]) if kind == "product" else c["type"]
        if kind == "linear":
            c["out"] = rng.choice([c["type"], "fp32"])
    else:
        c["H"], c["I"] = _width(rng, 256, 7168), _width(rng, 128, 2048)
        if kind == "ffn":
            c["save"] = rng.random() < 0.5
    return c


def _tokens(gen, T, width, type_, pad):
    """Normalised activations: unit variance, a few larger channels, in rows `pad` wider than they are."""
    x = torch.randn(T, width + pad, generator=gen, device="cuda")
    channel = torch.rand(width + pad, generator=gen, device="cuda")
    x = x * torch.where(channel < 0.01, 8.0, 1.0)
    return x.to(TYPES[type_])[:, :width]


def _weights(gen, out, inn, type_):
    return (torch.randn(out, inn, generator=gen, device="cuda") * inn**-0.5).to(TYPES[type_])


def _codes(w):
    """Codes and scales of rows, as a program makes them once for its weights."""
    scale = (w.double().abs().amax(1) / 127).float()
    q = (w.double() / scale.double()[:, None].clamp_min(1e-300)).round().clamp(-127, 127)
    return q.to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    kind, T, t = case["kind"], case["T"], case["type"]
    s = dict(case)
    if kind in ("product", "linear"):
        K, N = case["K"], case["N"]
        x = _tokens(gen, T, K, "fp32" if kind == "product" else t, case["pad"])
        s["w"], s["ws"] = _codes(_weights(gen, N, K, "fp32"))
        if kind == "product":
            q, s["xs"] = _codes(x)
            # codes in rows of their own stride
            s["q"] = torch.zeros(T, K + case["pad"], dtype=torch.int8, device="cuda")[:, :K].copy_(q)
        else:
            s["x"] = x
        return s
    H, I = case["H"], case["I"]
    s["x"] = _tokens(gen, T, H, t, case["pad"])
    w = [_weights(gen, I, H, t), _weights(gen, I, H, t), _weights(gen, H, I, t)]
    if kind == "int_ffn":
        for name, m in zip(("wg", "wu", "wd"), w):
            s[name], s[name + "s"] = _codes(m)
        return s
    s["wg"], s["wu"], s["wd"] = w
    if kind == "ffn_grad":
        x = s["x"].float()
        s["gu"] = torch.cat([x @ w[0].float().T, x @ w[1].float().T], 1).to(TYPES[t])
        s["dy"] = (torch.randn(T, H, generator=gen, device="cuda") * 0.25).to(TYPES[t])
    return s


def _quantise(x):
    """Row codes (as fp32 numbers) and scales; in 64 bits where a value lies next to a border between two codes."""
    scale = (x.double().abs().amax(1) / 127).float()
    q = (x.double() / scale.double()[:, None].clamp_min(1e-300)).round().clamp(-127, 127)
    return q.float(), scale


def _product(q, xs, w, ws):
    return (q @ w.float().T) * xs[:, None] * ws[None, :]


def _plain(s):
    kind = s["kind"]
    if kind == "product":
        return _product(s["q"].float(), s["xs"], s["w"], s["ws"]).to(TYPES[s["type"]])
    if kind == "linear":
        q, xs = _quantise(s["x"])
        return _product(q, xs, s["w"], s["ws"]).to(TYPES[s["out"]])
    t = TYPES[s["type"]]
    if kind == "int_ffn":
        q, xs = _quantise(s["x"])
        g, u = _product(q, xs, s["wg"], s["wgs"]), _product(q, xs, s["wu"], s["wus"])
        q, hs = _quantise(g / (1 + torch.exp(-g)) * u)
        return _product(q, hs, s["wd"], s["wds"]).to(t)
    x, wg, wu, wd = (s[n].float() for n in ("x", "wg", "wu", "wd"))
    if kind == "ffn":
        g, u = x @ wg.T, x @ wu.T
        y = ((g / (1 + torch.exp(-g)) * u) @ wd.T).to(t)
        return (y, torch.cat([g, u], 1).to(t)) if s["save"] else y
    I = s["I"]
    g, u, dy = s["gu"][:, :I].float(), s["gu"][:, I:].float(), s["dy"].float()
    sig = 1 / (1 + torch.exp(-g))
    dh = dy @ wd
    dg, du = dh * u * sig * (1 + g * (1 - sig)), dh * g * sig
    return {
        "dx": (dg @ wg + du @ wu).to(t),
        "dwg": (dg.T @ x).to(t),
        "dwu": (du.T @ x).to(t),
        "dwd": (dy.T @ (g * sig * u)).to(t),
    }


def _plan(s):
    """What a program keeps for calls of one size: the description, the workspace and the output buffers."""
    import lru_expert_cache_amd as ft

    kind, T, dev = s["kind"], s["T"], "cuda"
    dt = {"bf16": ft.FT_DT_BF16, "fp16": ft.FT_DT_F16, "fp32": ft.FT_DT_F32}
    p = {"ft": ft, "device": torch.cuda.current_device()}
    empty = lambda *n, type_=s["type"]: torch.empty(*n, dtype=TYPES[type_], device=dev)  # noqa: E731
    if kind in ("product", "linear"):
        K, N = s["K"], s["N"]
        p["q"], p["xs"] = s.get("q"), s.get("xs")
        if kind == "linear":
            p["dt"] = dt[s["type"]]
            p["q"], p["xs"] = torch.empty(T, K, dtype=torch.int8, device=dev), torch.empty(T, device=dev)
        out = s.get("out", s["type"])
        p["d"] = ft.make_int_matmul(T, K, N, dt[out], ld_x=p["q"].stride(0))
        p["work"] = torch.empty(ft.ft_moe_int_matmul_work(p["d"]), dtype=torch.uint8, device=dev)
        p["y"] = empty(T, N, type_=out)
        return p
    H, I = s["H"], s["I"]
    if kind == "int_ffn":
        p["d"] = ft.make_gated_ffn(dt[s["type"]], T, H, I, ld_x=s["x"].stride(0))
        p["work"] = torch.empty(ft.ft_moe_int_gated_ffn_work(p["d"]), dtype=torch.uint8, device=dev)
        p["y"] = empty(T, H)
        return p
    p["d"] = ft.make_gated_ffn(dt[s["type"]], T, H, I, ld_x=s["x"].stride(0))
    p["work"] = torch.empty(ft.ft_moe_gated_ffn_work(p["d"], kind == "ffn_grad"), dtype=torch.uint8, device=dev)
    if kind == "ffn":
        p["y"], p["gu"] = empty(T, H), empty(T, 2 * I) if s["save"] else None
    else:
        p["out"] = {"dx": torch.empty_like(s["x"]) if not s["pad"] else empty(T, H + s["pad"])[:, :H], "dwg": empty(I, H), "dwu": empty(I, H), "dwd": empty(H, I)}
    return p


def _kernels(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    ft, kind, d, work = p["ft"], s["kind"], p["d"], p["work"]
    # the calls' own default is the null stream; the inputs are made, and the results read, on the current one (its
    # handle: torch.cuda.current_stream() makes an object of it, for 2.8 us)
    stream = torch._C._cuda_getCurrentRawStream(p["device"])
    if kind in ("product", "linear"):
        if kind == "linear":
            ft.ft_moe_int_quantize(p["dt"], s["T"], s["K"], s["x"], p["q"], p["xs"], ld_x=s["x"].stride(0), stream=stream)
        ft.ft_moe_int_matmul(d, p["q"], p["xs"], s["w"], s["ws"], p["y"], work, stream)
        return p["y"]
    if kind == "int_ffn":
        ft.ft_moe_int_gated_ffn(d, s["x"], s["wg"], s["wgs"], s["wu"], s["wus"], s["wd"], s["wds"], p["y"], work, stream)
        return p["y"]
    if kind == "ffn":
        ft.ft_moe_gated_ffn_forward(d, s["x"], s["wg"], s["wu"], s["wd"], p["y"], p["gu"], work, stream)
        return (p["y"], p["gu"]) if s["save"] else p["y"]
    o = p["out"]
    ft.ft_moe_gated_ffn_backward(d, s["x"], s["wg"], s["wu"], s["wd"], s["gu"], s["dy"], o["dx"], o["dwg"], o["dwu"], o["dwd"], work, stream)
    return o


def run(state):
    return _kernels(state) if own else _plain(state)


def work(case):
    kind, T, b = case["kind"], case["T"], SIZE[case["type"]]
    if kind in ("product", "linear"):
        K, N = case["K"], case["N"]
        rows = T * K * b if kind == "linear" else T * K + 4 * T
        return {"bytes": rows + N * K + 4 * N + T * N * SIZE[case.get("out", case["type"])], "flops": 2 * T * N * K}
    H, I = case["H"], case["I"]
    if kind == "int_ffn":
        return {"bytes": 2 * T * H * b + 3 * H * I + 4 * (2 * I + H), "flops": 6 * T * H * I}
    if kind == "ffn":
        return {"bytes": (2 * T * H + 3 * H * I + (2 * T * I if case["save"] else 0)) * b, "flops": 6 * T * H * I}
    return {"bytes": (3 * T * H + 2 * T * I + 6 * H * I) * b, "flops": 12 * T * H * I}


def _codes64(v):
    """The definition of a row's codes, in 64 bits; the scale is a 32-bit number."""
    s = (v.double().abs().max(1, keepdim=True).values / 127).float().double()
    q = torch.where(s > 0, torch.round(v.double() / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(s))
    return torch.clamp(q, -127, 127), s


def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda n: s[n].to(torch.float64)  # noqa: E731
    mm = lambda a, b: torch.mm(a.contiguous(), b.transpose(0, 1).contiguous())  # noqa: E731
    kind = case["kind"]
    if kind in ("product", "linear"):
        q, xs = (f64("q"), f64("xs")[:, None]) if kind == "product" else _codes64(s["x"])
        return mm(q, f64("w")) * (xs * f64("ws")[None, :])
    if kind == "int_ffn":
        q, xs = _codes64(s["x"])
        g, u = (mm(q, f64(n)) * (xs * f64(n + "s")[None, :]) for n in ("wg", "wu"))
        h, hs = _codes64(g * torch.sigmoid(g) * u)
        return mm(h, f64("wd")) * (hs * f64("wds")[None, :])
    if kind == "ffn":
        g, u = mm(f64("x"), f64("wg")), mm(f64("x"), f64("wu"))
        y = mm(g * torch.sigmoid(g) * u, f64("wd"))
        return (y, torch.hstack([g, u])) if case["save"] else y
    g, u = torch.chunk(f64("gu"), 2, dim=1)
    p, dy, x = torch.sigmoid(g), f64("dy"), f64("x")
    dh = torch.mm(dy, f64("wd"))
    dg, du = dh * u * (p + g * p * torch.sigmoid(-g)), dh * (g * p)
    return {
        "dx": torch.mm(dg, f64("wg")) + torch.mm(du, f64("wu")),
        "dwg": mm(dg.transpose(0, 1), x.transpose(0, 1)),
        "dwu": mm(du.transpose(0, 1), x.transpose(0, 1)),
        "dwd": mm(dy.transpose(0, 1), (u * (g * p)).transpose(0, 1)),
    }
