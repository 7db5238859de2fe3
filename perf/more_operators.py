"""The operators around the feed-forward blocks and the router: cases, inputs, plain forms and exact values.

Four kinds of case:
  norm       s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, as 16-bit rows, as 8-bit codes with a scale per
             row, or both; the sum is kept as the residual of the next block
  norm_grad  its backward pass: gradients of x, of the residual and of the weight
  adapters   y = base + scale[a] (x A[a]^T) B[a]^T, a the adapter of each token (or none), base the shared projection
  balance    a router's step: top-k choice and weights, tokens per expert, the balance loss
             L = weight E sum_e f_e P_e (f_e: share of the choices that fall on e, P_e: its mean probability), and the
             gradient of L and of the routing weights with respect to the logits

Codes are given as the values they stand for.  Quantisation of a row: scale = fp32(max|row| / 127), code = row / scale
rounded to the nearest integer, ties to even.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


def listed():
    return [
        # one token on its way into an 8-bit block (the Qwen-A3B-shaped layer's width): latency
        {"name": "norm one token, 8 bit", "kind": "norm", "T": 1, "H": 2048, "type": "bf16", "res": "bf16", "y": False, "codes": True, "pad": 0},
        # a decode batch of the GLM-shaped layer: codes for the projection, 16-bit rows for router and adapters
        {"name": "norm decode batch, 8 bit", "kind": "norm", "T": 32, "H": 6144, "type": "bf16", "res": "bf16", "y": True, "codes": True, "pad": 0},
        # a prefill chunk of the DeepSeek-shaped layer, rows taken from a wider buffer
        {"name": "norm prefill, 8 bit", "kind": "norm", "T": 4096, "H": 7168, "type": "bf16", "res": "bf16", "y": False, "codes": True, "pad": 64},
        # forward pass of a training step with its residual stream in 32 bits
        {"name": "norm training forward", "kind": "norm", "T": 8192, "H": 7168, "type": "bf16", "res": "fp32", "y": True, "codes": False, "pad": 0},
        # gradients of a few rows (short fine-tuning samples)
        {"name": "norm gradient, few rows", "kind": "norm_grad", "T": 77, "H": 2048, "type": "fp16", "res": "fp16", "pad": 0},
        # gradients of a training step, the stream in 32 bits
        {"name": "norm gradient", "kind": "norm_grad", "T": 8192, "H": 7168, "type": "bf16", "res": "fp32", "pad": 0},
        # one request's token
        {"name": "adapters one token", "kind": "adapters", "T": 1, "K": 2048, "N": 2048, "R": 16, "n": 8, "type": "bf16", "base": "bf16", "out": "bf16", "mix": "decode", "pad": 0},
        # a decode batch, one token of each request, in no order
        {"name": "adapters decode batch", "kind": "adapters", "T": 32, "K": 6144, "N": 6144, "R": 16, "n": 32, "type": "bf16", "base": "bf16", "out": "bf16", "mix": "decode", "pad": 0},
        # prompts of several requests and single tokens of others, beside an 8-bit product with 32-bit results
        {"name": "adapters ragged batch", "kind": "adapters", "T": 1531, "K": 2048, "N": 5003, "R": 8, "n": 48, "type": "fp16", "base": "fp32", "out": "fp16", "mix": "both", "pad": 64},
        # a full prefill chunk of long prompts, adapters of a high rank
        {"name": "adapters prefill", "kind": "adapters", "T": 8192, "K": 7168, "N": 7168, "R": 64, "n": 16, "type": "bf16", "base": "bf16", "out": "bf16", "mix": "prompts", "pad": 0},
        # a router's step on one short sequence, some of it padding
        {"name": "balance short", "kind": "balance", "T": 509, "E": 128, "k": 8, "type": "fp32", "masked": 0.05, "pad": 0},
        # a router's step on a large batch of the DeepSeek-shaped layer
        {"name": "balance batch", "kind": "balance", "T": 32768, "E": 256, "k": 8, "type": "fp32", "masked": 0.0, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))


def _width(rng, lo, hi):
    """A width of a model: mostly multiples of 64, some of 16, now and then any number."""
    step = rng.choice([64, 64, 64, 64, 64, 64, 16, 16, 16, 1])
    return max(1, _log(rng, lo, hi) // step) * step


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_grad", "adapters", "adapters", "balance"])
    t = rng.choice(["bf16", "bf16", "fp16"])
    c = {"kind": kind, "T": _log(rng, 1, 8192), "type": t, "pad": rng.choice([0, 0, 64])}
    if kind in ("norm", "norm_grad"):
        c["type"] = t = rng.choice([t, t, t, "fp32"])
        c["H"], c["res"] = _width(rng, 256, 7168), rng.choice([t, "fp32"])
        if t == "fp32":  # twice the bytes
            c["T"] = max(1, c["T"] // 2)
        if kind == "norm":
            c["y"], c["codes"] = rng.choice([(True, False), (False, True), (True, True)])
    elif kind == "adapters":
        c["K"], c["N"] = _width(rng, 256, 7168), _width(rng, 256, 7168)
        c["R"], c["n"] = rng.choice([4, 8, 12, 16, 16, 24, 32, 64]), _log(rng, 1, 64)
        c["out"] = rng.choice([t, t, "fp32"])
        c["base"] = rng.choice([c["out"], "fp32", "none"])
        c["mix"] = "decode" if c["T"] <= 64 else rng.choice(["both", "prompts"])
        if "fp32" in (c["out"], c["base"]):
            c["T"] = max(1, c["T"] // 2)
    else:
        c["T"], c["E"] = _log(rng, 1, 32768), rng.choice([8, 16, 60, 64, 128, 160, 256])
        c["k"], c["type"] = rng.choice([1, 2, 4, 6, 8]), rng.choice(["fp32", "fp32", "bf16"])
        c["masked"] = rng.choice([0.0, 0.1])
    return c


def _rows(gen, T, width, type_, pad=0):
    """Activations: unit variance, a few larger channels, in rows `pad` wider than they are."""
    x = torch.randn(T, width + pad, generator=gen, device="cuda")
    channel = torch.rand(width + pad, generator=gen, device="cuda")
    x = x * torch.where(channel < 0.01, 8.0, 1.0)
    return x.to(TYPES[type_])[:, :width]


def _ids(gen, T, n, mix):
    """The adapter of each token, -1 for none (a fifth of the requests)."""
    # few adapters are asked for often, many seldom
    pick = lambda m: (n * torch.rand(m, generator=gen, device="cuda") ** 2).to(torch.int32).clamp(max=n - 1)  # noqa: E731
    one = torch.where(torch.rand(T, generator=gen, device="cuda") < 0.2, -1, pick(T))
    if mix == "decode":
        return one.to(torch.int32)
    # prompts of about 64 to 1000 tokens: a new one begins at some tokens
    starts = torch.rand(T, generator=gen, device="cuda") < 1.0 / (64 if mix == "both" else 500)
    ids = one[torch.cumsum(starts, 0).clamp(max=T - 1)]
    if mix == "both":  # the last quarter are single tokens
        ids[3 * T // 4 :] = one[3 * T // 4 :]
    return ids.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    kind, T, t = case["kind"], case["T"], case["type"]
    normal = lambda *n, scale=1.0: torch.randn(*n, generator=gen, device="cuda") * scale  # noqa: E731
    s = dict(case)
    if kind in ("norm", "norm_grad"):
        H, r = case["H"], TYPES[case["res"]]
        s["weight"] = (1.0 + normal(H, scale=0.2)).to(TYPES[t])
        if kind == "norm":
            s["x"] = _rows(gen, T, H, t, case["pad"])
            s["residual"] = (normal(T, H, scale=4.0)).to(r)
        else:
            s["sum"] = _rows(gen, T, H, case["res"], case["pad"])
            s["dy"] = normal(T, H, scale=0.25).to(TYPES[t])
            s["dsum"] = normal(T, H, scale=0.25).to(r)
    elif kind == "adapters":
        K, N, R, n = case["K"], case["N"], case["R"], case["n"]
        s["x"] = _rows(gen, T, K, t, case["pad"])
        s["a"], s["b"] = normal(n, R, K, scale=K**-0.5).to(TYPES[t]), normal(n, N, R, scale=R**-0.5).to(TYPES[t])
        s["scale"] = 0.25 + 0.5 * torch.rand(n, generator=gen, device="cuda")
        s["ids"] = _ids(gen, T, n, case["mix"])
        s["base_rows"] = None if case["base"] == "none" else normal(T, N).to(TYPES[case["base"]])
    else:
        E = case["E"]
        # some experts are asked for more than others
        s["logits"] = (normal(T, E + case["pad"], scale=1.5) + normal(E + case["pad"], scale=0.7)).to(TYPES[t])[:, :E]
        s["valid"] = (torch.rand(T, generator=gen, device="cuda") >= case["masked"]) if case["masked"] else None
        s["weight"] = 0.01
        s["dw"] = normal(T, case["k"], scale=0.25 / T)
        s["dloss"] = torch.ones((), device="cuda")
    return s


def _codes(v):
    """A row's codes as the values they stand for; v in 64 bits, since a value may lie next to a border."""
    scale = (v.abs().amax(1, keepdim=True) / 127).float()
    q = (v / scale.double().clamp_min(1e-300)).round().clamp(-127, 127)
    return q.float() * scale


def _plain_norm(s):
    f = torch.float64 if s["codes"] else torch.float32
    total = s["x"].to(f) + s["residual"].to(f)
    v = total * torch.rsqrt((total * total).mean(1, keepdim=True) + EPS) * s["weight"].to(f)
    out = {"sum": total.to(TYPES[s["res"]])}
    if s["y"]:
        out["y"] = v.to(TYPES[s["type"]])
    if s["codes"]:
        out["codes"] = _codes(v)
    return out


def _plain_norm_grad(s):
    x, dy, w = s["sum"].float(), s["dy"].float(), s["weight"].float()
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    n, g = x * r, dy * w
    ds = r * (g - n * (g * n).mean(1, keepdim=True)) + s["dsum"].float()
    out = {"dx": ds.to(TYPES[s["type"]]), "dweight": (dy * n).sum(0).to(TYPES[s["type"]])}
    if s["res"] != s["type"]:
        out["dresidual"] = ds
    return out


def _plain_adapters(s):
    T, R, n = s["T"], s["R"], s["n"]
    x, a, b = s["x"].float(), s["a"], s["b"]
    ids = s["ids"].long()
    some = ids >= 0
    at = ids.clamp(min=0)
    scale = torch.where(some, s["scale"][at], 0.0)
    if T <= n:  # each token's matrices, gathered
        h = torch.bmm(a[at].float(), x[:, :, None])
        y = torch.bmm(b[at].float(), h)[:, :, 0] * scale[:, None]
    else:  # every adapter's products, of which each token takes its own
        h = (x @ a.reshape(n * R, -1).float().T).view(T, n, R)
        mine = torch.arange(n, device=x.device)[None, :] == ids[:, None]
        h = torch.where(mine[:, :, None], h, 0.0) * scale[:, None, None]
        y = h.view(T, n * R) @ b.float().transpose(1, 2).reshape(n * R, -1)
    if s["base_rows"] is not None:
        y = y + s["base_rows"].float()
    return y.to(TYPES[s["out"]])


def _plain_balance(s):
    T, E, k = s["T"], s["E"], s["k"]
    z = s["logits"].float()
    valid = s["valid"] if s["valid"] is not None else torch.ones(T, dtype=torch.bool, device=z.device)
    on = valid[:, None]
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = torch.where(on, p / p.sum(1, keepdim=True), 0.0)
    top, order = torch.sort(z, dim=1, descending=True, stable=True)
    sel = order[:, :k]
    w = torch.exp(top[:, :k] - top[:, :1])
    w = torch.where(on, w / w.sum(1, keepdim=True), 0.0)
    chosen = torch.zeros(T, E, device=z.device).scatter_(1, sel, 1.0)
    counts = torch.where(on, chosen, 0.0).sum(0)
    tokens = valid.sum()
    c = s["weight"] * E / k * counts / (tokens.float() * tokens.float()).clamp(min=1.0)
    loss = (c.double() * p.double().sum(0)).sum().float()
    dz = s["dloss"] * p * (c - (p * c).sum(1, keepdim=True))
    dw = w * (s["dw"] - (w * s["dw"]).sum(1, keepdim=True))
    dz = dz.scatter_add(1, sel, dw)
    return {
        "sel": torch.where(on, sel, -1).to(torch.int32),
        "w": w,
        "counts": torch.cat([counts, tokens[None].float()]).to(torch.int32),
        "loss": loss[None],
        "dlogits": torch.where(on, dz, 0.0).to(TYPES[s["type"]]),
    }


def _plan(s):
    """What a program keeps for calls of one size: the description, the workspace and the output buffers."""
    import lru_expert_cache_amd as ft

    kind, T, t = s["kind"], s["T"], s["type"]
    dt = {"bf16": ft.FT_DT_BF16, "fp16": ft.FT_DT_F16, "fp32": ft.FT_DT_F32, "none": 0}
    empty = lambda *n, type_=t: torch.empty(*n, dtype=TYPES.get(type_, type_), device="cuda")  # noqa: E731
    p = {"ft": ft, "device": torch.cuda.current_device(), "out": {}, "work": None}
    o = p["out"]
    if kind == "norm":
        H = s["H"]
        p["d"] = ft.make_rms_norm(dt[t], T, H, EPS, residual_dtype=dt[s["res"]], ld_x=s["x"].stride(0))
        o["sum"] = empty(T, H, type_=s["res"])
        if s["y"]:
            o["y"] = empty(T, H)
        if s["codes"]:
            p["codes"], p["scale"] = empty(T, H, type_=torch.int8), empty(T, 1, type_=torch.float32)
        return p
    if kind == "norm_grad":
        H = s["H"]
        p["d"] = ft.make_rms_norm(dt[t], T, H, EPS, residual_dtype=dt[s["res"]], ld_sum=s["sum"].stride(0))
        o["dx"], o["dweight"] = empty(T, H), empty(H)
        if s["res"] != t:
            o["dresidual"] = empty(T, H, type_=s["res"])
        need = ft.ft_moe_rms_norm_work(p["d"])
    elif kind == "adapters":
        base = s["out"] if s["base"] == "none" else s["base"]
        p["d"] = ft.make_adapters(dt[t], T, s["K"], s["N"], s["R"], s["n"], base_dtype=dt[base], out_dtype=dt[s["out"]], ld_x=s["x"].stride(0))
        o["y"] = empty(T, s["N"], type_=s["out"])
        need = ft.ft_moe_adapters_work(p["d"])
    else:
        E, k = s["E"], s["k"]
        p["d"] = ft.make_balance(dt[t], T, E, k, s["weight"], ld_logits=s["logits"].stride(0))
        o["sel"], o["w"] = empty(T, k, type_=torch.int32), empty(T, k, type_=torch.float32)
        o["counts"], o["loss"] = empty(E + 1, type_=torch.int32), empty(1, type_=torch.float32)
        o["dlogits"] = torch.empty_strided((T, E), s["logits"].stride(), dtype=TYPES[t], device="cuda")
        need = ft.ft_moe_balance_work(p["d"])
    p["work"] = empty(max(need, 1), type_=torch.uint8)
    return p


def _kernels(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    ft, kind, d, work, o = p["ft"], s["kind"], p["d"], p["work"], p["out"]
    # the calls' own default is the null stream; the inputs are made, and the results read, on the current one
    stream = torch._C._cuda_getCurrentRawStream(p["device"])
    if kind == "norm":
        ft.ft_moe_rms_norm_forward(d, s["x"], s["residual"], s["weight"], o["sum"], o.get("y"), p.get("codes"), p.get("scale"), stream)
        return dict(o, codes=p["codes"] * p["scale"]) if s["codes"] else o
    if kind == "norm_grad":
        ft.ft_moe_rms_norm_backward(d, s["sum"], s["weight"], s["dy"], s["dsum"], o["dx"], o.get("dresidual"), o["dweight"], work, stream)
        return o
    if kind == "adapters":
        ft.ft_moe_adapters_apply(d, s["x"], s["ids"], s["a"], s["b"], s["scale"], s["base_rows"], o["y"], work, stream)
        return o["y"]
    ft.ft_moe_balance_forward(d, s["logits"], s["valid"], o["sel"], o["w"], o["counts"], o["loss"], work, stream)
    ft.ft_moe_balance_backward(d, s["logits"], s["valid"], o["sel"], o["w"], o["counts"], s["dw"], s["dloss"], o["dlogits"], stream)
    return o


def run(state):
    if own:
        return _kernels(state)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "adapters": _plain_adapters, "balance": _plain_balance}[state["kind"]](state)


def work(case):
    kind, T, b = case["kind"], case["T"], SIZE[case["type"]]
    if kind == "norm":
        H, r = case["H"], SIZE[case["res"]]
        each = b + 2 * r + (b if case["y"] else 0) + (1 if case["codes"] else 0)
        return {"bytes": T * H * each + b * H + (4 * T if case["codes"] else 0), "flops": 6 * T * H}
    if kind == "norm_grad":
        H, r = case["H"], SIZE[case["res"]]
        each = 2 * r + 2 * b + (r if case["res"] != case["type"] else 0)
        return {"bytes": T * H * each + 2 * b * H, "flops": 12 * T * H}
    if kind == "adapters":
        K, N, R = case["K"], case["N"], case["R"]
        base = 0 if case["base"] == "none" else SIZE[case["base"]]
        # the matrices of the adapters that the tokens can ask for
        return {
            "bytes": T * K * b + min(T, case["n"]) * R * (K + N) * b + T * N * (base + SIZE[case["out"]]) + 4 * T,
            "flops": 2 * T * R * (K + N),
        }
    E, k = case["E"], case["k"]
    # the logits are read by the forward pass and, the counts known, by the backward pass again
    return {"bytes": T * (3 * E * b + 20 * k) + 8 * E, "flops": T * (12 * E + 6 * k)}


def exact(case, seed):
    s = prepare(case, seed)
    kind, f64 = case["kind"], lambda n: s[n].to(torch.float64)  # noqa: E731
    if kind == "norm":
        total = torch.add(f64("x"), f64("residual"))
        v = total / torch.sqrt(total.square().mean(dim=-1) + EPS).unsqueeze(-1) * f64("weight")
        out = {"sum": total}
        if case["y"]:
            out["y"] = v
        if case["codes"]:
            scale = torch.div(v.abs().max(dim=1).values, 127.0).to(torch.float32).to(torch.float64).unsqueeze(1)
            out["codes"] = torch.round(v / scale) * scale
        return out
    if kind == "norm_grad":
        x, g = f64("sum"), f64("dy") * f64("weight")
        m = x.square().mean(dim=-1, keepdim=True) + EPS
        ds = g / m.sqrt() - x * torch.mean(g * x, dim=-1, keepdim=True) / (m * m.sqrt()) + f64("dsum")
        out = {"dx": ds, "dweight": torch.sum(f64("dy") * x / m.sqrt(), dim=0)}
        if case["res"] != case["type"]:
            out["dresidual"] = ds
        return out
    if kind == "adapters":
        y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
        if s["base_rows"] is not None:
            y += s["base_rows"]
        for a in range(case["n"]):
            at = torch.nonzero(s["ids"] == a)[:, 0]
            if at.numel():
                h = torch.mm(f64("x")[at], s["a"][a].double().t().contiguous())
                y[at] += float(s["scale"][a]) * torch.mm(h, s["b"][a].double().t().contiguous())
        return y
    T, E, k = case["T"], case["E"], case["k"]
    z, dw = f64("logits"), f64("dw")
    on = torch.ones(T, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"]
    p = torch.softmax(z, 1) * on[:, None]
    # the k largest, one after the other, the first of equal ones
    left, sel = z.clone(), []
    for _ in range(k):
        best = left.max(dim=1, keepdim=True).values
        at = torch.where(left == best, torch.arange(E, device="cuda"), E).min(dim=1).values
        sel.append(at)
        left[torch.arange(T, device="cuda"), at] = -math.inf
    sel = torch.stack(sel, 1)
    w = torch.softmax(torch.gather(z, 1, sel), 1) * on[:, None]
    counts = (torch.bincount(sel[on].reshape(-1), minlength=E)).double()
    tokens = max(1, int(on.sum()))
    c = s["weight"] * E * counts / (k * tokens)
    dz = p * (c - torch.mv(p, c)[:, None]) / tokens
    for i in range(k):
        dz[torch.arange(T, device="cuda"), sel[:, i]] += w[:, i] * (dw[:, i] - (w * dw).sum(1))
    return {
        "sel": torch.where(on[:, None], sel, -1).to(torch.int32),
        "w": w,
        "counts": torch.cat([counts, on.sum()[None].double()]).to(torch.int32),
        "loss": torch.dot(c, p.mean(0) * T / tokens)[None],
        "dlogits": dz * on[:, None],
    }
