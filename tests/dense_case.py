"""Inputs, 64-bit references and error bounds for the tests of the dense
feed-forward operators.

Every bound is elementwise and follows the operator's own steps: a 32-bit sum
of K products is off by at most (K + 2) 2^-23 times the sum of their
magnitudes (each addition rounds once, by at most one unit, whatever the
order), a rounding to a 16-bit type by half a unit relative to the value (plus
half its smallest subnormal), and an error of an intermediate is carried on by
the derivative's magnitude."""

import torch

import lru_expert_cache_amd as ft

TYPES = {"bf16": (torch.bfloat16, ft.FT_DT_BF16), "fp16": (torch.float16, ft.FT_DT_F16),
         "fp32": (torch.float32, ft.FT_DT_F32)}
U32 = 2.0**-23
SENTINEL = 7.25


def half_ulp(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the smallest subnormal."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def padded(rows, width, pad, dtype, fill=None, generator=None, scale=1.0):
    """A [rows, width] view of rows `pad` elements wider, between guard rows;
    filled with normal numbers, or with the sentinel."""
    buf = torch.full((rows + 2, width + pad), SENTINEL if fill is None else fill, dtype=torch.float32, device="cuda")
    if generator is not None:
        buf[1:rows + 1] = torch.randn(rows, width + pad, generator=generator, device="cuda") * scale
    buf = buf.to(dtype)
    return buf[1:rows + 1, :width], buf


def untouched(buf, rows, width):
    """Guard rows and padding columns still hold the sentinel."""
    s = torch.tensor(SENTINEL).to(buf.dtype).item()
    b = buf.float()
    return bool((b[0] == s).all() and (b[rows + 1:] == s).all() and (b[:, width:] == s).all())


def mm(a, b):
    return a.contiguous() @ b.contiguous()


def sum_error(a, b, k):
    """Bound on a 32-bit product of a [m, k] and b [k, n]."""
    return (k + 2) * U32 * mm(a.abs(), b.abs())


def sigmoid_error(g):
    # the exponent's argument rounds relative to itself, exp2, the sum and the reciprocal by a unit or two each
    return (g.abs() + 8) * U32


class Ffn:
    """One gated block in device memory, with output buffers."""

    def __init__(self, T, H, I, type_="bf16", pad=0, seed=0, wpad=0):
        self.T, self.H, self.I, self.pad, self.wpad = T, H, I, pad, wpad
        self.t, self.dt = TYPES[type_]
        g = torch.Generator(device="cuda")
        g.manual_seed(1000 + seed)
        self.x, _ = padded(T, H, pad, self.t, generator=g)
        self.wg, _ = padded(I, H, wpad, self.t, generator=g, scale=H**-0.5)
        self.wu, _ = padded(I, H, wpad, self.t, generator=g, scale=H**-0.5)
        self.wd, _ = padded(H, I, wpad, self.t, generator=g, scale=I**-0.5)
        self.dy, _ = padded(T, H, pad, self.t, generator=g)
        self.desc = ft.make_gated_ffn(self.dt, T, H, I, ld_x=H + pad, ld_y=H + pad, ld_gu=2 * I + pad, ld_w_in=H + wpad,
                                      ld_w_out=I + wpad)

    def work(self, backward):
        return torch.empty(ft.ft_moe_gated_ffn_work(self.desc, backward), dtype=torch.uint8, device="cuda")

    def forward(self, save=True, stream=None, work=None):
        y, yb = padded(self.T, self.H, self.pad, self.t)
        gu, gub = padded(self.T, 2 * self.I, self.pad, self.t)
        work = self.work(False) if work is None else work
        work.fill_(0xFF)  # NaN, should anything be read that was not written
        ft.ft_moe_gated_ffn_forward(self.desc, self.x, self.wg, self.wu, self.wd, y, gu if save else None, work, stream)
        torch.cuda.synchronize()
        assert untouched(yb, self.T, self.H) and untouched(gub, self.T, 2 * self.I)
        return y, gu

    def saved(self):
        """g and u as a forward pass leaves them, made by plain products."""
        gu, _ = padded(self.T, 2 * self.I, self.pad, self.t)
        gu.copy_(torch.cat([mm(self.x.double(), self.wg.double().T), mm(self.x.double(), self.wu.double().T)], 1).to(self.t))
        return gu

    def backward(self, gu, want_dx=True, want_dw=True, stream=None, work=None):
        t = self.t
        dx, dxb = padded(self.T, self.H, self.pad, t)
        dwg, gb = padded(self.I, self.H, self.wpad, t)
        dwu, ub = padded(self.I, self.H, self.wpad, t)
        dwd, db = padded(self.H, self.I, self.wpad, t)
        work = self.work(True) if work is None else work
        work.fill_(0xFF)
        w = (dwg, dwu, dwd) if want_dw else (None, None, None)
        ft.ft_moe_gated_ffn_backward(self.desc, self.x if want_dw else None, self.wg, self.wu, self.wd, gu, self.dy,
                                     dx if want_dx else None, *w, work, stream)
        torch.cuda.synchronize()
        assert untouched(dxb, self.T, self.H) and untouched(db, self.H, self.I)
        assert untouched(gb, self.I, self.H) and untouched(ub, self.I, self.H)
        return dx, dwg, dwu, dwd

    # 64-bit values and bounds
    def forward_reference(self):
        x, wg, wu, wd = (v.double() for v in (self.x, self.wg, self.wu, self.wd))
        e, z = half_ulp(self.t), tiny(self.t)
        g, u = mm(x, wg.T), mm(x, wu.T)
        dg, du = sum_error(x, wg.T, self.H), sum_error(x, wu.T, self.H)
        s = torch.sigmoid(g)
        h = g * s * u
        # |silu'| <= 1.1; first-order terms, doubled for the second order
        dh = 2 * (1.1 * dg * u.abs() + (g * s).abs() * du) + h.abs() * (sigmoid_error(g) + e + 4 * U32) + z
        y = mm(h, wd.T)
        dy = mm(dh, wd.abs().T) + sum_error(h, wd.T, self.I) * 2 + e * y.abs() * 1.01 + z
        gu = torch.cat([g, u], 1)
        dgu = torch.cat([dg, du], 1) * 1.01 + e * gu.abs() + z
        return (y, dy), (gu, dgu)

    def backward_reference(self, gu):
        x, wg, wu, wd, dy = (v.double() for v in (self.x, self.wg, self.wu, self.wd, self.dy))
        e, z, I, T = half_ulp(self.t), tiny(self.t), self.I, self.T
        g, u = gu[:, :I].double(), gu[:, I:].double()
        s = torch.sigmoid(g)
        se = sigmoid_error(g)
        dh, ddh = mm(dy, wd), sum_error(dy, wd, self.H)
        h, dhv = g * s * u, (g * s * u).abs() * (se + 4 * U32 + e) + z
        fg = u * s * (1 + g * (1 - s))
        # s and 1 - s are off by at most se (of one), which the bracket carries with |g|
        dfg = u.abs() * s * ((1 + g.abs()) * (2 * se + 8 * U32))
        dg, du = dh * fg, dh * g * s
        ddg = 2 * (ddh * fg.abs() + dh.abs() * dfg) + e * dg.abs() + z
        ddu = 2 * (ddh * (g * s).abs() + dh.abs() * (g * s).abs() * (se + 4 * U32)) + e * du.abs() + z

        def out(v, d):
            return v, d * 1.01 + e * v.abs() + z

        dx = out(mm(dg, wg) + mm(du, wu), mm(ddg, wg.abs()) + mm(ddu, wu.abs()) + 2 * sum_error(
            torch.cat([dg, du], 1), torch.cat([wg, wu], 0), 2 * I))
        dwg = out(mm(dg.T, x), mm(ddg.T, x.abs()) + 2 * sum_error(dg.T, x, T))
        dwu = out(mm(du.T, x), mm(ddu.T, x.abs()) + 2 * sum_error(du.T, x, T))
        dwd = out(mm(dy.T, h), mm(dy.abs().T, dhv) + 2 * sum_error(dy.T, h, T))
        return dx, dwg, dwu, dwd


def check(got, ref, what=""):
    v, bound = ref
    assert got.shape == v.shape
    if v.numel() == 0:
        return
    d = (got.double() - v).abs()
    assert torch.isfinite(d).all(), f"{what}: {int((~torch.isfinite(d)).sum())} values are not finite"
    worst = float((d / bound.clamp_min(1e-300)).max())
    assert worst <= 1.0, f"{what}: off by {worst:.3g} of the bound, at {int((d / bound).argmax())}"


def row_codes(x):
    """Codes and scales of rows by their definition, in 64 bits (finite rows)."""
    amax = x.double().abs().amax(1) if x.shape[0] else x.new_zeros(0).double()
    s = (amax / 127).float()
    q = torch.where(s[:, None] > 0, torch.round(x.double() / s.double()[:, None].clamp_min(1e-300)), 0.0)
    return q.clamp(-127, 127).to(torch.int8), s


def int_product_reference(q, xs, w, ws, out):
    """The product's value and bound: exact sums, three 32-bit roundings, one to the output's type."""
    v = mm(q.double(), w.double().T) * xs.double()[:, None] * ws.double()[None, :]
    return v, v.abs() * (4 * U32 + half_ulp(out)) + tiny(out)
