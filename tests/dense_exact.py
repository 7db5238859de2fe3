"""Inputs of the dense feed-forward operators whose results are known to the
last bit, for tests that compare bits: a term left out of a sum shows, whatever
the size.  The last terms along each K (where remainders lie) are never zero.

Operands are small multiples of powers of two with many zeros, so every sum is
an integer multiple of its smallest unit, below 2^24 units with all its terms
taken by magnitude: a 32-bit sum is exact in any order (`product` asserts it).
Gates are 18 or more, where 1 + e^-g rounds to 1 and the sigmoid is 1; below
-89, where e^-g overflows and it is 0; or 0, where it is 1/2: those reciprocals
are exact.  What is left are the operators' own roundings to their type, which
happen once and at known places: of the results, and of h and its gradients
where there are more than LO_FORWARD or LO_BACKWARD tokens.  Up to these the
values have up to 16 bits, so that both parts of them are needed.

Inputs are made on the CPU, so that tests without a GPU can look at the same
ones; references are plain products in the type `wide` on the inputs' device."""

import torch

import lru_expert_cache_amd as ft
from tests import dense_case as dc

# (tokens, hidden, inter): what the plan makes of those in TILED is pinned by the tests of the rules
SMALL = [(1, 2048, 768), (8, 264, 136), (9, 264, 136), (16, 512, 1000), (17, 264, 136), (33, 1000, 250), (64, 448, 320), (65, 320, 120), (77, 2048, 768), (300, 777, 901), (513, 136, 72)]
TILED = [(7990, 1983, 2043),  # 256 x 256 tiles in every form; odd widths, odd counts of K steps along H and T
         (8001, 2000, 1979),  # the same; an odd count along I, columns of H in whole groups of eight
         (4000, 7000, 2000),  # everything in whole groups; K of dh in parts
         (4097, 4000, 4100),  # K of dx in parts
         (8001, 1027, 2043),  # K of the weight gradients in parts
         (4090, 3901, 3907)]  # dx and the weight gradients in launches of their own, K whole
LO_FORWARD, LO_BACKWARD = 16, 64
PRODUCTS = [(5, 333, 77), (64, 2048, 257), (130, 1040, 333), (8001, 2003, 1921), (4090, 4083, 3901), (4096, 6144, 1024)]


def product(a, b, unit):
    """a b, exact: sums of magnitudes stay below 2^24 units."""
    v = dc.mm(a, b)
    assert float(dc.mm(a.abs(), b.abs()).max()) <= 2**24 * unit
    return v


def pick(g, rows, cols, density):
    """-1, 0 or 1."""
    r = torch.rand(rows, cols, generator=g)
    return (r < density / 2).float() - (r > 1 - density / 2).float()


def signs(g, *shape):
    """-1 or 1."""
    return torch.randint(2, shape, generator=g).float() * 2 - 1


def generator(seed):
    g = torch.Generator()
    g.manual_seed(4000 + seed)
    return g


class Values:
    """The numbers of one gated block, forward and backward, on the CPU in fp32."""

    def __init__(self, T, H, I, seed=0):
        self.T, self.H, self.I = T, H, I
        g = generator(seed)
        # sums of H products stay within 7 deviations of 14 / sqrt(2) or less, all through |r| <= 84
        p = min(0.5, 10 / H**0.5)
        self.x, self.wg, self.wu, self.wd = pick(g, T, H, p), pick(g, I, H, p), pick(g, I, H, p), pick(g, H, I, 0.3)
        # the first column decides the gate's sign: 144 or -172 beside the rest
        self.x[:, 0] = 1
        self.wg[:, 0] = torch.where(torch.rand(I, generator=g) < 0.7, 144.0, -172.0)
        self.wu[:, 0] = 0
        if H > 1:
            self.x[:, -1], self.wg[:, -1], self.wu[:, -1] = signs(g, T), signs(g, I), signs(g, I)
        self.wg[-1, 0], self.wd[:, -1] = 144, signs(g, H)
        self.wd /= 32
        # backward: gates and ups of their own, as a caller's gu holds them; dh like the sums above
        self.gu = torch.empty(T, 2 * I)
        few = T <= LO_BACKWARD
        self.gu[:, :I] = torch.tensor([25.0, 37.0, 0.0, -128.0] if few else [32.0, 32.0, 0.0, -128.0])[torch.randint(4, (T, I), generator=g)]
        ups = torch.arange(-31.0, 32.0) if few else torch.tensor([1.0, -1.0, 2.0, -2.0, 0.0])
        self.gu[:, I:] = ups[torch.randint(len(ups), (T, I), generator=g)]
        self.dy, self.bd = pick(g, T, H, p), pick(g, H, I, p)
        self.bx, self.bg, self.bu = pick(g, T, H, 0.3) / 8, pick(g, I, H, 0.3), pick(g, I, H, 0.3) / 4
        for at in ((slice(None), I - 1), (-1, slice(0, I))):  # the last term of dx, of the weight gradients
            self.gu[at] = 32
        self.gu[:, 2 * I - 1], self.gu[-1, I:] = signs(g, T), signs(g, I)
        self.bg[-1], self.bu[-1], self.bx[-1] = signs(g, H), signs(g, H) / 4, signs(g, H) / 8
        self.dy[:, -1], self.bd[-1] = signs(g, T), signs(g, I)

    def to(self, device, wide):
        for n in ("x", "wg", "wu", "wd", "gu", "dy", "bd", "bx", "bg", "bu"):
            setattr(self, n, getattr(self, n).to(device, wide))
        return self

    def forward(self, t):
        """y and gu rounded to t, and what they are made of."""
        g, u = product(self.x, self.wg.T, 1), product(self.x, self.wu.T, 1)
        assert bool(((g >= 32) & (g <= 256) | (g <= -89) & (g >= -256)).all()) and float(u.abs().max()) <= 112
        h = torch.where(g > 0, g * u, 0)
        h = h if self.T <= LO_FORWARD else h.to(t).to(g.dtype)
        y = product(h, self.wd.T, 2**-5)
        return y.to(t), torch.cat([g, u], 1).to(t), h, y

    def dgu(self, dh):
        g, u = self.gu[:, :self.I], self.gu[:, self.I:]
        s = torch.where(g > 0, 1.0, torch.where(g < 0, 0.0, 0.5)).to(g.dtype)
        return dh * u * s, dh * g * s, g * s * u

    def backward(self, t):
        """dx, dwg, dwu, dwd before they are rounded to t, and what they are made of."""
        dh = product(self.dy, self.bd, 1)
        assert float(dh.abs().max()) <= 112  # dg in halves, du in 32nds: eight bits each
        dg, du, h = self.dgu(dh)
        for v in (dg, du, h):
            hi = v.to(torch.bfloat16).to(v.dtype)
            lo = (v - hi).to(torch.bfloat16).to(v.dtype)
            assert torch.equal(v, hi + lo if self.T <= LO_BACKWARD else hi)
        dx = product(torch.cat([dg, du], 1), torch.cat([self.bg, self.bu], 0), 0.5)
        return dx, product(dg.T, self.bx, 2**-4), product(du.T, self.bx, 2**-3), product(self.dy.T, h, 1), (dg, du, h)


class Block(dc.Ffn):
    """These numbers as a block in device memory, with the calls of the other tests; rows `pad` elements wider."""

    def __init__(self, v, type_, backward, pad=0, wpad=0):
        self.T, self.H, self.I, self.pad, self.wpad = v.T, v.H, v.I, pad, wpad
        self.t, self.dt = dc.TYPES[type_]
        T, H, I = v.T, v.H, v.I

        def put(m, pad):
            view, _ = dc.padded(*m.shape, pad, self.t)
            return view.copy_(m)

        self.x = put(v.bx if backward else v.x, pad)
        self.wg, self.wu = (put(m, wpad) for m in ((v.bg, v.bu) if backward else (v.wg, v.wu)))
        self.wd = put(v.bd if backward else v.wd, wpad)
        self.dy, self.gu = put(v.dy, pad), put(v.gu, pad)
        self.desc = ft.make_gated_ffn(self.dt, T, H, I, ld_x=H + pad, ld_y=H + pad, ld_gu=2 * I + pad, ld_w_in=H + wpad,
                                      ld_w_out=I + wpad)


class IntValues:
    """The 8-bit block: tokens that are their own codes (their largest is 127, so the scale is 1)."""

    def __init__(self, T, H, I, seed=0):
        self.T, self.H, self.I = T, H, I
        g = generator(100 + seed)
        p = min(0.5, 10 / H**0.5)
        self.x, self.wg, self.wu, self.wd = pick(g, T, H, p), pick(g, I, H, p), pick(g, I, H, p), pick(g, H, I, 0.3)
        self.x[:, 0] = 127
        self.wg[:, 0] = torch.where(torch.rand(I, generator=g) < 0.7, 1.0, -2.0)  # gates of 127 or -254 beside the rest
        self.wu[:, 0] = 0
        self.x[:, -1], self.wg[:, -1], self.wu[:, -1], self.wd[:, -1] = signs(g, T), signs(g, I), signs(g, I), signs(g, H)
        self.wg[-1, 0] = 1
        self.down = torch.pow(2.0, torch.randint(-8, -2, (H,), generator=g).float())

    def to(self, device, wide):
        for n in ("x", "wg", "wu", "wd"):
            setattr(self, n, getattr(self, n).to(device, wide))
        self.down = self.down.to(device)
        return self

    def forward(self, t):
        g, u = product(self.x, self.wg.T, 1), product(self.x, self.wu.T, 1)
        assert bool(((g >= 18) | (g <= -89)).all())
        h = torch.where(g > 0, g * u, 0)
        q, hs = dc.row_codes(h.float())
        s = product(q.to(self.wd.dtype), self.wd.T, 1)
        return (s.float() * hs[:, None] * self.down[None, :]).to(t), q, hs, s
