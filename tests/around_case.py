"""Inputs, 64-bit references and error bounds for the tests of the norm, the
adapters and the router's balance.

Every bound is elementwise and counts roundings: E = 2^-24 is half a unit of a
32-bit number relative to its value, half_ulp(t) that of the output's type
(plus half its smallest subnormal), and an error of an intermediate is carried
on by the derivative's magnitude."""

import torch

import lru_expert_cache_amd as ft
from tests.dense_case import TYPES, check, half_ulp, padded, tiny, untouched  # noqa: F401

E = 2.0**-24
DT = {name: dt for name, (_, dt) in TYPES.items()}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rounded(v, t, also=0.0):
    """Bound of a value that is rounded to t at the end, off by `also` before."""
    return also + (half_ulp(t) * 1.001) * (v.abs() + also) + tiny(t)


# ------------------------------------------------------------ norm
class Norm:
    """A norm's inputs and output buffers in rows `pad` wider than they are, between guard rows."""

    def __init__(self, rows, cols, type_="bf16", res=None, pad=0, eps=1e-6, seed=0):
        self.rows, self.cols, self.pad, self.eps = rows, cols, pad, eps
        self.t, self.r = TYPES[type_][0], TYPES[res or type_][0]
        g = gen(7000 + seed)
        self.x, _ = padded(rows, cols, pad, self.t, generator=g)
        self.residual, _ = padded(rows, cols, pad, self.r, generator=g, scale=3.0)
        self.weight = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(self.t)
        self.dy, _ = padded(rows, cols, pad, self.t, generator=g)
        self.dsum, _ = padded(rows, cols, pad, self.r, generator=g)
        self.s, _ = padded(rows, cols, pad, self.r, generator=g, scale=2.0)  # the backward pass's sum
        ld = cols + pad
        self.d = ft.make_rms_norm(DT[type_], rows, cols, eps, residual_dtype=DT[res or type_], ld_x=ld, ld_residual=ld,
                                  ld_sum=ld, ld_y=ld, ld_codes=ld)

    def forward(self, residual=True, sum_=True, y=True, codes=True, stream=None):
        R, C, P = self.rows, self.cols, self.pad
        out = {"sum": padded(R, C, P, self.r), "y": padded(R, C, P, self.t), "codes": padded(R, C, P, torch.int8)}
        scale = torch.full((R + 2,), 7.25, device="cuda")
        ft.ft_moe_rms_norm_forward(self.d, self.x, self.residual if residual else None, self.weight,
                                   out["sum"][0] if sum_ else None, out["y"][0] if y else None,
                                   out["codes"][0] if codes else None, scale[1:] if codes else None, stream)
        torch.cuda.synchronize()
        for name, wanted in (("sum", sum_), ("y", y), ("codes", codes)):
            assert untouched(out[name][1], R if wanted else 0, C), name
        assert scale[0] == 7.25 and scale[R + 1] == 7.25
        return {"sum": out["sum"][0], "y": out["y"][0], "codes": out["codes"][0], "scale": scale[1:R + 1]}

    def forward_reference(self, residual=True):
        s = self.x.double() + (self.residual.double() if residual else 0.0)
        v = s / torch.sqrt((s * s).mean(1, keepdim=True) + self.eps) * self.weight.double()
        scale = (v.abs().amax(1) / 127).float()
        live = (scale > 0)[:, None]
        codes = torch.where(live, torch.round(v / torch.where(live, scale[:, None].double(), 1.0)), 0.0)
        # up to four roundings to 32 bits before the last one
        return {"sum": (s, rounded(s, self.r, E * s.abs())), "y": (v, rounded(v, self.t, 4 * E * v.abs())),
                "codes": codes.clamp(-127, 127).to(torch.int8), "scale": scale}

    def work(self):
        return torch.empty(max(1, ft.ft_moe_rms_norm_work(self.d)), dtype=torch.uint8, device="cuda").fill_(0xFF)

    def backward(self, dsum=True, dx=True, dresidual=True, dweight=True, stream=None, work=None):
        R, C, P = self.rows, self.cols, self.pad
        out = {"dx": padded(R, C, P, self.t), "dresidual": padded(R, C, P, self.r)}
        dw = torch.full((C + 2,), 7.25, device="cuda").to(self.t)
        ft.ft_moe_rms_norm_backward(self.d, self.s, self.weight, self.dy, self.dsum if dsum else None,
                                    out["dx"][0] if dx else None, out["dresidual"][0] if dresidual else None,
                                    dw[1:] if dweight else None, self.work() if work is None else work, stream)
        torch.cuda.synchronize()
        for name, wanted in (("dx", dx), ("dresidual", dresidual)):
            assert untouched(out[name][1], R if wanted else 0, C), name
        assert dw[0] == 7.25 and dw[C + 1] == 7.25
        return {"dx": out["dx"][0], "dresidual": out["dresidual"][0], "dweight": dw[1:C + 1]}

    def backward_reference(self, dsum=True):
        s, dy, w = self.s.double(), self.dy.double(), self.weight.double()
        r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + self.eps)
        n, g = s * r, dy * w
        m = (g * n).mean(1, keepdim=True)
        more = self.dsum.double() if dsum else 0.0
        ds = r * (g - n * m) + more
        # g, r, m, n, the difference and its product with r round once or twice each; m carries g's rounding; then the sum
        off = E * 1.01 * (r * (6 * g.abs() + 6 * (n * m).abs() + n.abs() * (g * n).abs().mean(1, keepdim=True)) + ds.abs())
        dw = (dy * n).sum(0)
        # two roundings of n, and one addition for each row and each group of rows on the way
        offw = (self.rows + 90) * E * (dy * n).abs().sum(0)
        return {"dx": (ds, rounded(ds, self.t, off)), "dresidual": (ds, rounded(ds, self.r, off)),
                "dweight": (dw, rounded(dw, self.t, offw))}


# ------------------------------------------------------------ adapters
class Adapters:
    def __init__(self, tokens, in_, out, rank, count, type_="bf16", base="same", out_type=None, pad=0, wpad=0, seed=0,
                 ids=None, scale=True):
        self.tokens, self.out, self.rank, self.count, self.pad = tokens, out, rank, count, pad
        self.t, self.o = TYPES[type_][0], TYPES[out_type or type_][0]
        base_type = (out_type or type_) if base in ("same", None) else base
        g = gen(8000 + seed)
        self.x, _ = padded(tokens, in_, pad, self.t, generator=g)
        self.a = padded(count * rank, in_, wpad, self.t, generator=g, scale=in_**-0.5)[0]
        self.b = padded(count * out, rank, wpad, self.t, generator=g, scale=rank**-0.5)[0]
        self.scale = 0.5 + torch.rand(count, generator=g, device="cuda") if scale else None
        self.base = None if base is None else padded(tokens, out, pad, TYPES[base_type][0], generator=g)[0]
        self.ids = (torch.randint(-1, count, (tokens,), generator=g, device="cuda") if ids is None
                    else torch.as_tensor(ids, device="cuda")).to(torch.int32)
        self.d = ft.make_adapters(DT[type_], tokens, in_, out, rank, count, base_dtype=DT[base_type],
                                  out_dtype=DT[out_type or type_], ld_x=in_ + pad, ld_a=in_ + wpad, ld_b=rank + wpad,
                                  ld_base=out + pad, ld_y=out + pad)

    def work(self):
        return torch.empty(ft.ft_moe_adapters_work(self.d), dtype=torch.uint8, device="cuda").fill_(0xFF)

    def apply(self, stream=None, work=None):
        y, yb = padded(self.tokens, self.out, self.pad, self.o)
        ft.ft_moe_adapters_apply(self.d, self.x, self.ids, self.a, self.b, self.scale, self.base, y,
                                 self.work() if work is None else work, stream)
        torch.cuda.synchronize()
        assert untouched(yb, self.tokens, self.out)
        return y

    def reference(self):
        T, N, R, n, K = self.tokens, self.out, self.rank, self.count, self.x.shape[1]
        v = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        off = torch.zeros_like(v)
        for i in range(n):
            at = torch.nonzero(self.ids == i)[:, 0]
            if not at.numel():
                continue
            a, b = self.a[i * R:(i + 1) * R].double(), self.b[i * N:(i + 1) * N].double()
            x = self.x[at].double()
            s = 1.0 if self.scale is None else float(self.scale[i])
            h, hm = x @ a.T.contiguous(), x.abs() @ a.abs().T.contiguous()
            # a 32-bit sum rounds once for each term (by a unit at most) and twice more; in two 16-bit parts a bf16
            # value keeps 16 bits and more, an fp16 one 22; the second sum has up to three parts of each term
            dh = (K + 2) * 2 * E * hm + h.abs() * 2.0**-17
            m = b.abs().T.contiguous()
            v[at] = s * (h @ b.T.contiguous())
            off[at] = abs(s) * (dh @ m + (3 * R + 4) * 2 * E * ((h.abs() + dh) @ m))
        if self.base is not None:
            v = v + self.base.double()
        return v, rounded(v, self.o, off + E * v.abs())


# ------------------------------------------------------------ balance
class Balance:
    def __init__(self, tokens, experts, top_k, type_="fp32", weight=0.01, masked=0.2, pad=0, seed=0, ties=False):
        self.tokens, self.experts, self.top_k, self.pad = tokens, experts, top_k, pad
        self.t, self.weight = TYPES[type_][0], weight
        g = gen(9000 + seed)
        self.z, _ = padded(tokens, experts, pad, self.t, generator=g, scale=2.0)
        if ties:  # few different values
            self.z.copy_((self.z.float() * 2).round() / 2)
        self.valid = torch.rand(tokens, generator=g, device="cuda") >= masked if masked else None
        self.dw = torch.randn(tokens, top_k, generator=g, device="cuda")
        self.dloss = torch.full((1,), 1.7, device="cuda")
        self.d = ft.make_balance(DT[type_], tokens, experts, top_k, weight, ld_logits=experts + pad)

    def work(self):
        return torch.empty(ft.ft_moe_balance_work(self.d), dtype=torch.uint8, device="cuda").fill_(0xFF)

    def forward(self, stream=None, work=None):
        T, k = self.tokens, self.top_k
        sel, w = torch.full((T + 2, k), -77, dtype=torch.int32, device="cuda"), torch.full((T + 2, k), 7.25, device="cuda")
        counts, loss = torch.full((self.experts + 3,), -77, dtype=torch.int32, device="cuda"), torch.full((3,), 7.25, device="cuda")
        ft.ft_moe_balance_forward(self.d, self.z, self.valid, sel[1:], w[1:], counts[1:], loss[1:],
                                  self.work() if work is None else work, stream)
        torch.cuda.synchronize()
        assert (sel[0] == -77).all() and (sel[T + 1] == -77).all() and (w[0] == 7.25).all() and (w[T + 1] == 7.25).all()
        assert counts[0] == -77 and counts[-1] == -77 and loss[0] == 7.25 and loss[2] == 7.25
        return {"sel": sel[1:T + 1], "w": w[1:T + 1], "counts": counts[1:-1], "loss": loss[1:2]}

    def backward(self, f, dw=True, dloss=True, stream=None):
        dz, zb = padded(self.tokens, self.experts, self.pad, self.t)
        ft.ft_moe_balance_backward(self.d, self.z, self.valid, f["sel"] if dw else None, f["w"] if dw else None,
                                   f["counts"], self.dw if dw else None, self.dloss if dloss else None, dz, stream)
        torch.cuda.synchronize()
        assert untouched(zb, self.tokens, self.experts)
        return dz

    def reference(self):
        """Values and bounds of sel, w, counts, loss and of dlogits (finite logits and -inf)."""
        T, N, k = self.tokens, self.experts, self.top_k
        z = self.z.double()
        inf = torch.finfo(torch.float64).max
        on = torch.ones(T, dtype=torch.bool, device="cuda") if self.valid is None else self.valid.bool()
        on = on & ~(z == -torch.inf).all(1)
        z = torch.where(on[:, None], z, 0.0)
        d = (z - z.amax(1, keepdim=True)).clamp_min(-inf)
        p = torch.softmax(z, 1)
        # an exponent's argument rounds once or twice relative to itself (times log2 e), exp by a unit or two; the sum
        # carries its terms' errors, and rounds for each of a lane's 8 terms and 6 steps between lanes
        near = torch.where(p > 0, p * d.abs().clamp_max(1e4), 0.0).sum(1, keepdim=True)
        ep = p * (3 * d.abs().clamp_max(1e4) + 3 * near + 40) * E
        order = torch.sort(z, dim=1, descending=True, stable=True)
        sel, top = order.indices[:, :k], order.values[:, :k]
        some = on[:, None] & (top > -torch.inf)
        dt = (top - top[:, :1]).clamp_min(-inf)
        w = torch.softmax(top, 1)
        near = torch.where(w > 0, w * dt.abs().clamp_max(1e4), 0.0).sum(1, keepdim=True)
        ew = w * (3 * dt.abs().clamp_max(1e4) + 3 * near + 40) * E + 2.0**-149
        counts = torch.zeros(N, dtype=torch.float64, device="cuda").index_add_(0, sel[some], torch.ones_like(top[some]))
        V = int(on.sum())
        c = self.weight * N * counts / (k * max(V, 1) ** 2)
        p, ep = p * on[:, None], ep * on[:, None]
        loss = (c * p.sum(0)).sum()
        # a lane adds its tokens one after the other, then the waves; the rest is done in 64 bits
        eloss = (c.abs() * (ep.sum(0) + (T / 256 + 24) * E * p.sum(0))).sum() + 2 * E * loss.abs() + 2.0**-149
        self.dref = (z, p, ep, torch.where(some, w, 0.0), ew, c, sel, some, on)
        return {"sel": torch.where(some, sel, -1).to(torch.int32), "w": (torch.where(some, w, 0.0), ew), "loss": (loss[None], eloss[None]),
                "counts": torch.cat([counts, on.sum()[None].double()]).to(torch.int32)}

    def backward_reference(self, dw=True, dloss=True):
        self.reference()
        _, p, ep, w, ew, c, sel, some, on = self.dref
        g = abs(float(self.dloss)) if dloss else 1.0
        sign = -1.0 if dloss and float(self.dloss) < 0 else 1.0
        s = (p * c).sum(1, keepdim=True)
        es = (ep * c.abs()).sum(1, keepdim=True) + 20 * E * (p * c.abs()).sum(1, keepdim=True)
        dz = sign * g * p * (c - s)
        off = g * (ep * (c - s).abs() + p * (3 * E * c.abs() + es)) * 1.01 + 4 * E * dz.abs()
        if dw:
            v = self.dw.double()
            m = (w * v).sum(1, keepdim=True)
            em = ((ew + 10 * E * w) * v.abs()).sum(1, keepdim=True)
            one = torch.where(some, w * (v - m), 0.0)
            eone = torch.where(some, ew * (v - m).abs() + w * em + 4 * E * w * (v.abs() + m.abs()), 0.0)
            dz = dz.scatter_add(1, sel, one)
            off = off.scatter_add(1, sel, eone) + 2 * E * dz.abs()
        dz, off = dz * on[:, None], off * on[:, None]
        return dz, rounded(dz, self.t, off)
