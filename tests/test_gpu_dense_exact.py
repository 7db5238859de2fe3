"""Dense feed-forward operators on the GPU, bit for bit: inputs whose results have known bits (dense_exact.py), in every
form, on each kernel and tile size."""

import pytest
import torch

import lru_expert_cache_amd as ft
from tests import dense_case as dc
from tests import dense_exact as de

pytestmark = pytest.mark.gpu

BOTH = [(s, t) for s in de.SMALL for t in ("bf16", "fp16")] + [(s, ("bf16", "fp16")[i % 2]) for i, s in enumerate(de.TILED)]
BOTH += [(de.TILED[0], "fp16"), (de.TILED[2], "fp16")]


def same(got, want, what):
    wrong = got != want
    assert got.shape == want.shape and not bool(wrong.any()), \
        f"{what}: {int(wrong.sum())} of {wrong.numel()} differ, first at {wrong.nonzero()[0].tolist()}"


@pytest.mark.parametrize("size,type_", BOTH)
def test_forward(size, type_):
    v = de.Values(*size).to("cuda", torch.float64)
    b = de.Block(v, type_, False)
    want_y, want_gu, _, _ = v.forward(b.t)
    y, gu = b.forward()
    same(gu, want_gu, "gu")
    same(y, want_y, "y")


@pytest.mark.parametrize("size,type_", BOTH)
def test_backward(size, type_):
    v = de.Values(*size).to("cuda", torch.float64)
    b = de.Block(v, type_, True)
    want = v.backward(b.t)
    for kw in (dict(), dict(want_dw=False), dict(want_dx=False)):  # together (and in one launch where that is the plan), alone
        got = b.backward(b.gu, **kw)
        for i, name in enumerate(("dx", "dwg", "dwu", "dwd")):
            if kw.get("want_dx" if i == 0 else "want_dw", True):
                same(got[i], want[i].to(b.t), f"{name} {kw}")


@pytest.mark.parametrize("type_", ["bf16", "fp16"])
@pytest.mark.parametrize("size", [s for s in de.SMALL] + de.TILED[:2])
def test_int_gated_ffn(size, type_):
    v = de.IntValues(*size).to("cuda", torch.float64)
    t, dt = dc.TYPES[type_]
    T, H, I = size
    want = v.forward(t)[0]
    one = torch.ones(I, device="cuda")
    y, yb = dc.padded(T, H, 0, t)
    d = ft.make_gated_ffn(dt, T, H, I)
    work = torch.empty(ft.ft_moe_int_gated_ffn_work(d), dtype=torch.uint8, device="cuda").fill_(0xFF)
    ft.ft_moe_int_gated_ffn(d, v.x.to(t), v.wg.to(torch.int8), one, v.wu.to(torch.int8), one, v.wd.to(torch.int8), v.down, y, work)
    torch.cuda.synchronize()
    assert dc.untouched(yb, T, H)
    same(y, want, "y")


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("size", de.PRODUCTS)
def test_int_matmul(size, out):
    """Scales that are powers of two: the exact sum rounds to fp32, then to the output's type."""
    T, K, N = size
    t, dt = dc.TYPES[out]
    g = de.generator(7)
    q, w = (torch.randint(-127, 128, (n, K), generator=g, dtype=torch.int8).cuda() for n in (T, N))
    xs, ws = (torch.pow(2.0, torch.randint(-12, -6, (n,), generator=g).float()).cuda() for n in (T, N))
    y, yb = dc.padded(T, N, 0, t)
    d = ft.make_int_matmul(T, K, N, dt)
    work = torch.empty(ft.ft_moe_int_matmul_work(d), dtype=torch.uint8, device="cuda").fill_(0xFF)
    ft.ft_moe_int_matmul(d, q, xs, w, ws, y, work)
    torch.cuda.synchronize()
    assert dc.untouched(yb, T, N)
    same(y, (dc.mm(q.double(), w.double().T).float() * xs[:, None] * ws[None, :]).to(t), "y")


def off_grid(m, off):
    """The same rows from an address `off` elements past a 16-byte one, as far apart."""
    ld = m.stride(0) if m.dim() == 2 else 1
    flat = torch.zeros(m.shape[0] * ld + off + 64, dtype=m.dtype, device=m.device)
    start = off + (-flat.data_ptr() // m.element_size()) % (16 // m.element_size())
    return flat.as_strided(m.shape, m.stride(), start).copy_(m)


@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("name", ["x", "w"])
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
def test_int_matmul_off_the_grid(T, name, out):
    """Codes at addresses that are no multiples of 16 bytes, rows of whole pieces and not: the general kernel, in all
    its output types."""
    t, dt = dc.TYPES[out]
    g = de.generator(8)
    for K, N in ((256, 130), (250, 77)):
        q, w = (torch.randint(-127, 128, (n, K), generator=g, dtype=torch.int8).cuda() for n in (T, N))
        xs, ws = (torch.pow(2.0, torch.randint(-12, -6, (n,), generator=g).float()).cuda() for n in (T, N))
        a = {"x": q, "w": w}
        a[name] = off_grid(a[name], 3)
        assert a[name].data_ptr() % 16
        y, yb = dc.padded(T, N, 5, t)
        d = ft.make_int_matmul(T, K, N, dt, ld_y=N + 5)
        work = torch.empty(ft.ft_moe_int_matmul_work(d), dtype=torch.uint8, device="cuda").fill_(0xFF)
        ft.ft_moe_int_matmul(d, a["x"], xs, a["w"], ws, y, work)
        torch.cuda.synchronize()
        assert dc.untouched(yb, T, N)
        same(y, (dc.mm(q.double(), w.double().T).float() * xs[:, None] * ws[None, :]).to(t), f"y {K} {N}")


@pytest.mark.parametrize("size", [(3, 64, 48), (70, 64, 48), (70, 61, 43), (200, 320, 136)])
@pytest.mark.parametrize("name", ["x", "wg", "wu", "wd", "all"])
@pytest.mark.parametrize("type_", ["bf16", "fp16"])
def test_int_block_off_the_grid(size, name, type_):
    v = de.IntValues(*size).to("cuda", torch.float64)
    t, dt = dc.TYPES[type_]
    T, H, I = size
    one = torch.ones(I, device="cuda")
    a = {"x": v.x.to(t), "wg": v.wg.to(torch.int8), "wu": v.wu.to(torch.int8), "wd": v.wd.to(torch.int8)}
    for n in a if name == "all" else (name,):
        a[n] = off_grid(a[n], 1)
        assert a[n].data_ptr() % 16
    y, yb = dc.padded(T, H, 0, t)
    d = ft.make_gated_ffn(dt, T, H, I)
    work = torch.empty(ft.ft_moe_int_gated_ffn_work(d), dtype=torch.uint8, device="cuda").fill_(0xFF)
    ft.ft_moe_int_gated_ffn(d, a["x"], a["wg"], one, a["wu"], one, a["wd"], v.down, y, work)
    torch.cuda.synchronize()
    assert dc.untouched(yb, T, H)
    same(y, v.forward(t)[0], "y")


@pytest.mark.parametrize("size", [(3, 64, 48), (70, 61, 43), (200, 320, 136)])
@pytest.mark.parametrize("type_", ["bf16", "fp16"])
def test_block_off_the_grid(size, type_):
    """Each operand, results and saved values among them, and then all."""
    v = de.Values(*size).to("cuda", torch.float64)
    T, H, I = size
    t, dt = dc.TYPES[type_]
    desc = ft.make_gated_ffn(dt, T, H, I)
    forward = [(m.to(t)) for m in (v.x, v.wg, v.wu, v.wd)]
    backward = [m.to(t) for m in (v.bx, v.bg, v.bu, v.bd, v.gu, v.dy)]
    want_f, want_b = v.forward(t)[:2], [m.to(t) for m in v.backward(t)[:4]]
    new = lambda r, c, off: off_grid(torch.zeros(r, c, dtype=t, device="cuda"), off)  # noqa: E731
    for at in range(7):
        a = [off_grid(m, 1) if at in (i, 6) else m for i, m in enumerate(forward)]
        out = [new(T, n, 3 if at in (4 + i, 6) else 0) for i, n in enumerate((H, 2 * I))]
        work = torch.empty(ft.ft_moe_gated_ffn_work(desc), dtype=torch.uint8, device="cuda").fill_(0xFF)
        ft.ft_moe_gated_ffn_forward(desc, *a, *out, work)
        for got, want, what in zip(out, want_f, ("y", "gu")):
            same(got, want, f"{what}, {at} off")
    for at in range(11):
        a = [off_grid(m, 5) if at in (i, 10) else m for i, m in enumerate(backward)]
        out = [new(*s, 1 if at in (6 + i, 10) else 0) for i, s in enumerate(((T, H), (I, H), (I, H), (H, I)))]
        work = torch.empty(ft.ft_moe_gated_ffn_work(desc, True), dtype=torch.uint8, device="cuda").fill_(0xFF)
        ft.ft_moe_gated_ffn_backward(desc, *a, *out, work)
        for got, want, what in zip(out, want_b, ("dx", "dwg", "dwu", "dwd")):
            same(got, want, f"{what}, {at} off")


def test_one_token_that_holds_a_nan_or_an_infinity():
    for bad in ("nan", "inf", "-inf"):
        f = dc.Ffn(1, 256, 192)
        f.x[0, 3] = float(bad)
        assert bool((f.wg[:, 3] < 0).any()) and bool((f.wg[:, 3] > 0).any())  # infinite gates of both signs: -inf * 0 is NaN
        y, gu = f.forward()
        assert bool(torch.isnan(y).all()) and not bool(torch.isfinite(gu).any()), bad


@pytest.mark.parametrize("T", [6, 18])
def test_range_of_fp16(T):
    """h is rounded to the block's type (a few tokens' keep what that leaves off): up to fp16's largest number it gives a finite y; beyond, its token's y is not
    finite, and the other tokens keep their bits."""
    H, I, n = 32, 16, T // 6
    t, dt = dc.TYPES["fp16"]
    x, wg, wu, wd = (torch.zeros(n, m, dtype=t, device="cuda") for n, m in ((T, H), (I, H), (I, H), (H, I)))
    x[:, 0] = 1
    x[:, 1] = torch.tensor([65.5, 0.5, 65.5, 66.0, 65.5, -66.0] * n)  # u: h = 65500, which rounds to 65504, or 66000
    wg[:, 0], wu[:, 1] = 1000, 1
    wd[torch.arange(H), torch.arange(H) % I] = 2.0**-8
    y, gu = torch.empty(T, H, dtype=t, device="cuda"), torch.empty(T, 2 * I, dtype=t, device="cuda")
    d = ft.make_gated_ffn(dt, T, H, I)
    work = torch.empty(ft.ft_moe_gated_ffn_work(d), dtype=torch.uint8, device="cuda")
    ft.ft_moe_gated_ffn_forward(d, x, wg, wu, wd, y, gu, work)
    want = torch.tensor([65504.0, 500.0, 65504.0, 0.0, 65504.0, 0.0] * n, device="cuda") * 2.0**-8
    keep = want > 0
    same(gu, torch.cat([torch.full((T, I), 1000.0), x[:, 1:2].cpu().expand(T, I)], 1).to(t).cuda(), "gu")
    same(y[keep], want[keep, None].expand(-1, H).to(t), "y")
    assert not bool(torch.isfinite(y[~keep]).any())


def pick(g, density, *shape):
    """-1, 0 or 1 on the GPU, in bf16 (for matrices too large to make on the CPU)."""
    r = torch.randint(0, 1 << 14, shape, generator=g, device="cuda", dtype=torch.int16)
    at = int(density / 2 * (1 << 14))
    return (r < at).to(torch.bfloat16) - (r >= (1 << 14) - at).to(torch.bfloat16)


def gates(g, T, I, on):
    """g of 32 (a share `on`), else -128; u of 1 or -1: what the backward pass is given."""
    gu = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
    gu[:, :I] = torch.where(torch.randint(0, 1 << 14, (T, I), generator=g, device="cuda", dtype=torch.int16) < int(on * (1 << 14)), 32.0, -128.0)
    gu[:, I:] = torch.where(torch.randint(0, 2, (T, I), generator=g, device="cuda", dtype=torch.int16) > 0, 1.0, -1.0)
    return gu


def ends(n, far):
    return (slice(0, far), slice(n - far, n))


@pytest.mark.parametrize("T", [2, 70])
def test_weights_past_32_bits(T):
    """Weight matrices of more than 4 GB, forward and backward: results at both ends, bit for bit."""
    H, I, far, t = 8192, 270_000, 2000, torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    x, dy = pick(g, 0.1, T, H), pick(g, 0.1, T, H)
    wg, wu, wd = pick(g, 0.1, I, H), pick(g, 0.1, I, H), pick(g, 0.1, H, I)
    assert wg.numel() * 2 > 1 << 32
    x[:, 0], wu[:, 0], wd[:, -1], wd[-1] = 1, 0, 1, 1
    wg[:, 0] = -172  # closed gates, but for one in fifty (the last among them)
    wg[::50, 0] = wg[-1, 0] = 144
    d = ft.make_gated_ffn(ft.FT_DT_BF16, T, H, I)
    work = torch.empty(ft.ft_moe_gated_ffn_work(d), dtype=torch.uint8, device="cuda").fill_(0xFF)
    y, gu = torch.empty(T, H, dtype=t, device="cuda"), torch.empty(T, 2 * I, dtype=t, device="cuda")
    ft.ft_moe_gated_ffn_forward(d, x, wg, wu, wd, y, gu, work)
    for part in ends(I, far):
        same(gu[:, part], de.product(x.double(), wg[part].double().T, 1).to(t), "g")
        same(gu[:, I:][:, part], de.product(x.double(), wu[part].double().T, 1).to(t), "u")
    v, u = gu[:, :I].double(), gu[:, I:].double()
    assert bool(((v >= 32) & (v <= 256) | (v <= -89) & (v >= -256)).all()) and float(u.abs().max()) <= 112
    h = torch.where(v > 0, v * u, 0)
    h = h if T <= de.LO_FORWARD else h.to(t)
    for part in ends(H, far):
        same(y[:, part], de.product(h.double(), wd[part].double().T, 1).to(t), "y")
    del y, v, u, h, work
    gu = gates(g, T, I, 0.1)
    work = torch.empty(ft.ft_moe_gated_ffn_work(d, True), dtype=torch.uint8, device="cuda").fill_(0xFF)
    dx, dwg, dwu, dwd = (torch.empty_like(m) for m in (x, wg, wu, wd))
    wg[:, 0] = 1
    ft.ft_moe_gated_ffn_backward(d, x, wg, wu, wd, gu, dy, dx, dwg, dwu, dwd, work)
    dh = de.product(dy.double(), wd.double(), 1)
    assert float(dh.abs().max()) <= 256
    v, u = gu[:, :I].double(), gu[:, I:].double()
    s = (v > 0).double()
    dg, du, h = dh * u * s, dh * v * s, v * s * u
    sums = de.product(dg, wg.double(), 1) + de.product(du, wu.double(), 32)
    assert float((dc.mm(dg.abs(), wg.double().abs()) + dc.mm(du.abs(), wu.double().abs())).max()) <= 2**24
    same(dx, sums.to(t), "dx")
    for part in ends(I, far):
        same(dwg[part], de.product(dg[:, part].T, x.double(), 1).to(t), "dwg")
        same(dwu[part], de.product(du[:, part].T, x.double(), 32).to(t), "dwu")
    for part in ends(H, far):
        same(dwd[part], de.product(dy[:, part].double().T, h, 32).to(t), "dwd")


def test_tokens_past_32_bits():
    """So many tokens that every tensor of theirs passes 4 GB: the ends of what has their rows, the weight gradients
    whole, bit for bit; and the 8-bit block, whose last tokens have the bits that they have alone."""
    T, H, I, far, t = 2_200_000, 1024, 1000, 2000, torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(22)
    x, wg, wu, wd = pick(g, 0.1, T, H), pick(g, 0.1, I, H), pick(g, 0.1, I, H), pick(g, 0.3, H, I)
    assert T * min(H, I) * 2 > 1 << 32
    x[:, 0], wu[:, 0] = 1, 0
    wg[:, 0] = -172
    wg[::4, 0] = 144
    d = ft.make_gated_ffn(ft.FT_DT_BF16, T, H, I)
    work = torch.empty(ft.ft_moe_gated_ffn_work(d), dtype=torch.uint8, device="cuda").fill_(0xFF)
    y, gu = torch.empty(T, H, dtype=t, device="cuda"), torch.empty(T, 2 * I, dtype=t, device="cuda")
    ft.ft_moe_gated_ffn_forward(d, x, wg, wu, wd, y, gu, work)
    for part in ends(T, far):
        v, u = (de.product(x[part].double(), w.double().T, 1) for w in (wg, wu))
        same(gu[part], torch.cat([v, u], 1).to(t), "gu")
        assert bool(((v >= 32) & (v <= 256) | (v <= -89) & (v >= -256)).all()) and float(u.abs().max()) <= 112
        h = torch.where(v > 0, v * u, 0).to(t).double()
        same(y[part], de.product(h, wd.double().T, 1).to(t), "y")
    del gu, work
    # 8 bit: the tokens as their own rows, weights as codes
    one, down = torch.ones(I, device="cuda"), torch.ones(H, device="cuda")
    codes = (wg.clamp(-100, 100).to(torch.int8), one, wu.to(torch.int8), one, wd.to(torch.int8), down)
    y8 = torch.empty(T, H, dtype=t, device="cuda")
    work = torch.empty(ft.ft_moe_int_gated_ffn_work(d), dtype=torch.uint8, device="cuda").fill_(0xFF)
    ft.ft_moe_int_gated_ffn(d, x, *codes, y8, work)
    for part in (slice(0, 100), slice(T - 100, T)):
        few = ft.make_gated_ffn(ft.FT_DT_BF16, 100, H, I)
        alone = torch.empty(100, H, dtype=t, device="cuda")
        ft.ft_moe_int_gated_ffn(few, x[part], *codes, alone, work)
        same(y8[part], alone, "y, 8 bit")
    del y8, work
    dy, gu = y, gates(g, T, I, 0.25)
    dy.copy_(pick(g, 0.1, T, H))
    work = torch.empty(ft.ft_moe_gated_ffn_work(d, True), dtype=torch.uint8, device="cuda").fill_(0xFF)
    dx, dwg, dwu, dwd = (torch.empty_like(m) for m in (x, wg, wu, wd))
    wg[:, 0] = 1
    ft.ft_moe_gated_ffn_backward(d, x, wg, wu, wd, gu, dy, dx, dwg, dwu, dwd, work)
    sums = [torch.zeros(*s, dtype=torch.float64, device="cuda") for s in ((I, H), (I, H), (H, I))]
    tops = [torch.zeros_like(s) for s in sums]
    step = 110_000
    for r in range(0, T, step):
        part = slice(r, r + step)
        dh = de.product(dy[part].double(), wd.double(), 1)
        assert float(dh.abs().max()) <= 256
        v, u = gu[part, :I].double(), gu[part, I:].double()
        s = (v > 0).double()
        dg, du, h = dh * u * s, dh * v * s, v * s * u
        for total, top, a, b in zip(sums, tops, (dg, du, dy[part].double()), (x[part].double(), x[part].double(), h)):
            total += dc.mm(a.T, b)
            top += dc.mm(a.T.abs(), b.abs())
        if r in (0, T - step):
            assert float((dc.mm(dg.abs(), wg.double().abs()) + dc.mm(du.abs(), wu.double().abs())).max()) <= 2**24
            same(dx[part], (dc.mm(dg, wg.double()) + dc.mm(du, wu.double())).to(t), "dx")
    for got, total, top, unit, what in zip((dwg, dwu, dwd), sums, tops, (1, 32, 32), ("dwg", "dwu", "dwd")):
        assert float(top.max()) <= 2**24 * unit
        same(got, total.to(t), what)


def few(T, H, I, type_, seed, off=0):
    """Normal numbers, all operands `off` elements past a 16-byte address."""
    f = dc.Ffn(T, H, I, type_, seed=seed)
    for n in ("x", "wg", "wu", "wd", "dy") if off else ():
        setattr(f, n, off_grid(getattr(f, n), off))
    return f


FEW = [(1, 256, 128, 0), (1, 512, 768, 0), (3, 129, 67, 0), (8, 320, 136, 0), (8, 200, 128, 3), (2, 64, 1, 0), (9, 256, 128, 0), (16, 320, 200, 0), (13, 129, 67, 0), (16, 72, 61, 1)]


@pytest.mark.parametrize("type_", ["bf16", "fp16"])
@pytest.mark.parametrize("size", FEW)
def test_few_tokens_are_rounded_once_forward(size, type_):
    """y of up to 16 tokens is off by its own rounding and what 32-bit sums lose: h keeps both its 16-bit parts, so that
    it is off by half a unit of half a unit (and half the smallest number)."""
    for seed in range(5):
        f = few(*size[:3], type_, seed, size[3])
        y, _ = f.forward()
        x, wg, wu, wd = (v.double() for v in (f.x, f.wg, f.wu, f.wd))
        e, z = dc.half_ulp(f.t), dc.tiny(f.t)
        g, u = dc.mm(x, wg.T), dc.mm(x, wu.T)
        eg, eu, s = dc.sum_error(x, wg.T, f.H), dc.sum_error(x, wu.T, f.H), torch.sigmoid(g)
        h = g * s * u
        eh = 2 * (1.1 * eg * u.abs() + (g * s).abs() * eu) + h.abs() * (dc.sigmoid_error(g) + e * e + 4 * dc.U32) + z
        v = dc.mm(h, wd.T)
        dc.check(y, (v, (dc.mm(eh, wd.abs().T) + 2 * dc.sum_error(h, wd.T, 2 * f.I)) * 1.01 + e * v.abs() + z), f"y {seed}")


@pytest.mark.parametrize("type_", ["bf16", "fp16"])
@pytest.mark.parametrize("size", FEW + [(33, 130, 72, 0), (64, 256, 200, 0), (64, 72, 61, 1)])
def test_few_tokens_are_rounded_once_backward(size, type_):
    """The same of the gradients of up to 64 tokens: of dg, du and h."""
    for seed in range(3):
        f = few(*size[:3], type_, seed, size[3])
        gu = f.saved()
        got = f.backward(gu)
        x, wg, wu, wd, dy = (v.double() for v in (f.x, f.wg, f.wu, f.wd, f.dy))
        e, z, I, T = dc.half_ulp(f.t), dc.tiny(f.t), f.I, f.T
        g, u = gu[:, :I].double(), gu[:, I:].double()
        s, se = torch.sigmoid(g), dc.sigmoid_error(g)
        dh, edh = dc.mm(dy, wd), dc.sum_error(dy, wd, f.H)
        h = g * s * u
        eh = h.abs() * (se + 4 * dc.U32 + e * e) + z
        fg = u * s * (1 + g * (1 - s))
        efg = u.abs() * s * ((1 + g.abs()) * (2 * se + 8 * dc.U32))
        dg, du = dh * fg, dh * g * s
        edg = 2 * (edh * fg.abs() + dh.abs() * efg) + e * e * dg.abs() + z
        edu = 2 * (edh * (g * s).abs() + dh.abs() * (g * s).abs() * (se + 4 * dc.U32)) + e * e * du.abs() + z
        both, w = torch.cat([dg, du], 1), torch.cat([wg, wu], 0)
        want = ((dc.mm(both, w), dc.mm(torch.cat([edg, edu], 1), w.abs()) + 2 * dc.sum_error(both, w, 4 * I)),
                (dc.mm(dg.T, x), dc.mm(edg.T, x.abs()) + 2 * dc.sum_error(dg.T, x, 2 * T)),
                (dc.mm(du.T, x), dc.mm(edu.T, x.abs()) + 2 * dc.sum_error(du.T, x, 2 * T)),
                (dc.mm(dy.T, h), dc.mm(dy.abs().T, eh) + 2 * dc.sum_error(dy.T, h, 2 * T)))
        for m, (v, err), name in zip(got, want, ("dx", "dwg", "dwu", "dwd")):
            dc.check(m, (v, err * 1.01 + e * v.abs() + z), f"{name} {seed}")
