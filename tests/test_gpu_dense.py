"""Dense feed-forward operators on the GPU against 64-bit references: the gated
block and its gradients, 8-bit rows, the 8-bit product and the 8-bit block, over
lengths, odd sizes, strides and types; then the calls as a program makes them
(streams, graphs, scratch memory, forward with backward)."""

import pytest
import torch

import lru_expert_cache_amd as ft
from tests import dense_case as dc

pytestmark = pytest.mark.gpu

# (tokens, hidden, inter, row padding of tokens, of weights)
SIZES = [
    (1, 1, 1, 0, 0),
    (3, 7, 5, 0, 0),
    (1, 256, 128, 0, 0),
    (2, 2048, 768, 0, 0),
    (5, 264, 136, 8, 0),
    (16, 512, 2048, 0, 0),
    (17, 1024, 96, 0, 8),
    (31, 200, 72, 3, 0),       # token rows off the 16-byte grid
    (33, 129, 67, 0, 0),       # everything odd
    (64, 448, 320, 0, 64),
    (70, 1000, 250, 0, 0),     # inter not a multiple of 4
    (77, 2048, 768, 0, 0),
    (128, 64, 1032, 64, 0),
    (257, 384, 640, 0, 8),
    (300, 2048, 40, 0, 5),     # weight rows off the grid
    (513, 136, 72, 0, 0),
    (1100, 512, 768, 0, 0),
]


@pytest.mark.parametrize("type_", ["bf16", "fp16"])
@pytest.mark.parametrize("size", SIZES)
def test_forward(size, type_):
    T, H, I, pad, wpad = size
    f = dc.Ffn(T, H, I, type_, pad, wpad=wpad)
    (y, gu), (ry, rgu) = f.forward(), f.forward_reference()
    dc.check(y, ry, "y")
    dc.check(gu, rgu, "gu")
    y2, _ = f.forward(save=False)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("type_", ["bf16", "fp16"])
@pytest.mark.parametrize("size", SIZES)
def test_backward(size, type_):
    T, H, I, pad, wpad = size
    f = dc.Ffn(T, H, I, type_, pad, wpad=wpad)
    gu = f.saved()
    got = f.backward(gu)
    for v, r, name in zip(got, f.backward_reference(gu), ("dx", "dwg", "dwu", "dwd")):
        dc.check(v, r, name)
    # each half alone gives the same bits
    dx = f.backward(gu, want_dw=False)[0]
    assert torch.equal(dx, got[0])
    assert all(torch.equal(a, b) for a, b in zip(f.backward(gu, want_dx=False)[1:], got[1:]))


@pytest.mark.parametrize("size", [(4096, 2048, 768), (2049, 1024, 2048)])
def test_large(size):
    f = dc.Ffn(*size)
    (y, gu), (ry, rgu) = f.forward(), f.forward_reference()
    dc.check(y, ry, "y")
    dc.check(gu, rgu, "gu")
    for v, r, name in zip(f.backward(gu), f.backward_reference(gu), ("dx", "dwg", "dwu", "dwd")):
        dc.check(v, r, name)


def test_gradients_follow_differences():
    """The gradients of sum(y * dy) against central differences of a 64-bit block, along random directions."""
    f = dc.Ffn(6, 40, 24, "fp16", seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    gu = f.saved()
    dx, dwg, dwu, dwd = f.backward(gu)

    def loss(x, wg, wu, wd):
        a = x @ wg.T
        return ((a * torch.sigmoid(a) * (x @ wu.T)) @ wd.T * f.dy.double()).sum()

    at = [v.double() for v in (f.x, f.wg, f.wu, f.wd)]
    refs = f.backward_reference(gu)
    for i, grad in enumerate((dx, dwg, dwu, dwd)):
        v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 2.0**-12
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + step * v, at[i] - step * v
        difference = (loss(*hi) - loss(*lo)) / (2 * step)
        # the kernel's bound; the saved g and u are rounded, which moves the 64-bit gradient by as much again as one
        # more rounding of every intermediate (factor 4); differences of a smooth function at 2^-12 add 2^-24 times its
        # third derivative, of the order of the gradient
        bound = 4 * (refs[i][1] * v.abs()).sum() + 1e-5 * (refs[i][0] * v).abs().sum()
        assert (difference - (grad.double() * v).sum()).abs() <= bound


def test_no_tokens():
    f = dc.Ffn(0, 64, 32)
    f.forward()
    _, dwg, dwu, dwd = f.backward(torch.empty(0, 64, dtype=f.t, device="cuda"))
    assert all(bool((v == 0).all()) for v in (dwg, dwu, dwd))


def test_rows_are_independent():
    """A token that holds a NaN or an infinity leaves the other tokens' bits alone."""
    for T in (1, 9, 40, 200):
        f = dc.Ffn(T, 256, 192)
        y, gu = f.forward()
        at = T // 2
        f.x[at, 3] = float("nan") if T > 1 else float("inf")
        y2, gu2 = f.forward()
        assert bool(torch.isnan(y2[at]).all()) or T == 1
        keep = torch.arange(T, device="cuda") != at
        assert torch.equal(y[keep], y2[keep]) and torch.equal(gu[keep], gu2[keep])


def test_large_magnitudes():
    """Gates far outside exp's range: silu(-large) is -0, silu(large) is its argument."""
    f = dc.Ffn(8, 64, 32, "bf16")
    f.wg.mul_(1000)
    (y, gu), (ry, rgu) = f.forward(), f.forward_reference()
    dc.check(y, ry, "y")
    for v, r, name in zip(f.backward(gu), f.backward_reference(gu), ("dx", "dwg", "dwu", "dwd")):
        dc.check(v, r, name)


# ---------------------------------------------------------------- 8 bit
QUANT = [(1, 1, 0), (3, 17, 0), (2, 2048, 0), (33, 7168, 0), (5, 6144, 64), (64, 130, 3), (1021, 2048, 0), (7, 20000, 8)]


@pytest.mark.parametrize("type_", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("size", QUANT)
def test_quantize(size, type_):
    rows, cols, pad = size
    t, dt = dc.TYPES[type_]
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    x, _ = dc.padded(rows, cols, pad, t, generator=g)
    if rows > 2:
        x[1] = 0
        x[2] = x[2] * 2.0**-12
    codes = torch.full((rows + 1, cols + pad), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((rows + 1,), dc.SENTINEL, device="cuda")
    ft.ft_moe_int_quantize(dt, rows, cols, x, codes, scale, ld_x=cols + pad, ld_codes=cols + pad)
    q, s = dc.row_codes(x)
    assert torch.equal(scale[:rows].cpu(), s.cpu()) and float(scale[rows]) == dc.SENTINEL
    assert torch.equal(codes[:rows, :cols], q)
    assert bool((codes[:rows, cols:] == 99).all()) and bool((codes[rows] == 99).all())


def test_quantize_ties_and_extremes():
    """Quotients that lie half-way go to the even code; subnormal, huge and non-finite rows."""
    n = torch.arange(-127, 127, device="cuda").float() + 0.5
    rows = [torch.cat([n * 2.0**e, torch.tensor([127.0 * 2.0**e], device="cuda")]) for e in (0, -8, -140, -149 + 1, 100, 120)]
    # a third of a unit in the last place beside a tie: scale 1/3 of a power of two
    rows.append(torch.cat([n / 3, torch.tensor([127 / 3], device="cuda")]))
    x = torch.stack(rows)
    codes, scale = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(x.shape[0], device="cuda")
    ft.ft_moe_int_quantize(ft.FT_DT_F32, *x.shape, x, codes, scale)
    q, s = dc.row_codes(x)
    assert torch.equal(scale, s) and torch.equal(codes, q)
    assert torch.equal(codes[0, :-1].float(), torch.round(n))
    x = torch.randn(4, 64, device="cuda")
    x[0, 5], x[1, 6], x[2, 7] = float("inf"), float("nan"), -float("inf")
    x[3] = 1e-45  # its scale is below the smallest number
    codes, scale = torch.full(x.shape, 5, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    ft.ft_moe_int_quantize(ft.FT_DT_F32, 4, 64, x, codes, scale)
    assert bool(torch.isnan(scale[:3]).all()) and float(scale[3]) == 0 and bool((codes == 0).all())


# (tokens, in, out, padding of token codes, of weights, of results)
PRODUCTS = [(1, 1, 1, 0, 0, 0), (1, 7168, 512, 0, 0, 0), (2, 100, 33, 0, 0, 0), (7, 256, 100, 16, 0, 0),
            (16, 2048, 1000, 0, 0, 0), (17, 640, 130, 0, 16, 2), (33, 4096, 256, 0, 0, 0), (64, 96, 520, 0, 0, 0),
            (100, 1040, 257, 0, 0, 0), (130, 333, 77, 1, 3, 5), (257, 512, 384, 0, 0, 8), (1021, 2048, 603, 0, 0, 0),
            (700, 131071, 40, 1, 1, 0)]


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("size", PRODUCTS)
def test_int_matmul(size, out):
    T, K, N, px, pw, py = size
    t, dt = dc.TYPES[out]
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    q = torch.randint(-127, 128, (T, K + px), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K + pw), generator=g, device="cuda", dtype=torch.int8)
    if T > 2:
        q[1] = 127  # the largest sums
    w[0] = 127
    xs, ws = (torch.rand(n, generator=g, device="cuda") * 1e-3 for n in (T, N))
    y, yb = dc.padded(T, N, py, t)
    d = ft.make_int_matmul(T, K, N, dt, ld_x=K + px, ld_w=K + pw, ld_y=N + py)
    work = torch.empty(ft.ft_moe_int_matmul_work(d), dtype=torch.uint8, device="cuda").fill_(0xFF)
    ft.ft_moe_int_matmul(d, q, xs, w, ws, y, work)
    torch.cuda.synchronize()
    assert dc.untouched(yb, T, N)
    dc.check(y, dc.int_product_reference(q[:, :K], xs, w[:, :K], ws, t), "y")


def _int_block(T, H, I, type_, pad=0, wpad=0, seed=0):
    f = dc.Ffn(T, H, I, type_, pad, seed=seed)
    codes = []
    for m in (f.wg, f.wu, f.wd):
        q, s = dc.row_codes(m)
        wide = torch.full((q.shape[0], q.shape[1] + wpad), 77, dtype=torch.int8, device="cuda")
        wide[:, :q.shape[1]] = q
        codes += [wide, s]
    d = ft.make_gated_ffn(f.dt, T, H, I, ld_x=H + pad, ld_y=H + pad, ld_w_in=H + wpad, ld_w_out=I + wpad)
    return f, codes, d


def _run_int_block(f, codes, d, stream=None):
    y, yb = dc.padded(f.T, f.H, f.pad, f.t)
    work = torch.empty(ft.ft_moe_int_gated_ffn_work(d), dtype=torch.uint8, device="cuda").fill_(0xFF)
    ft.ft_moe_int_gated_ffn(d, f.x, *codes, y, work, stream)
    torch.cuda.synchronize()
    assert dc.untouched(yb, f.T, f.H)
    return y


@pytest.mark.parametrize("type_", ["bf16", "fp16"])
@pytest.mark.parametrize("size", [s for s in SIZES if s[0] != 0])
def test_int_gated_ffn(size, type_):
    T, H, I, pad, wpad = size
    f, codes, d = _int_block(T, H, I, type_, pad, wpad)
    y = _run_int_block(f, codes, d)
    (wg, sg, wu, su, wd, sd) = (c[:, :w] if c.dim() == 2 else c for c, w in zip(codes, (H, 0, H, 0, I, 0)))
    q, xs = dc.row_codes(f.x)
    g, eg = dc.int_product_reference(q, xs, wg, sg, torch.float32)
    u, eu = dc.int_product_reference(q, xs, wu, su, torch.float32)
    h = g * torch.sigmoid(g) * u
    eh = 2 * (1.1 * eg * u.abs() + (g * torch.sigmoid(g)).abs() * eu) + h.abs() * (dc.sigmoid_error(g) + 4 * dc.U32)
    hq, hs = dc.row_codes(h.float())
    # the scale moves with the row's largest value; a code may differ where its quotient is that near to a tie
    es = eh.max(1).values / 127 + hs * 2 * dc.U32
    quot = (h / hs.double()[:, None].clamp_min(1e-300)).clamp(-127, 127)
    near = ((quot.abs() % 1) - 0.5).abs() * hs.double()[:, None] <= eh + quot.abs() * es[:, None] + hs.double()[:, None] * dc.U32
    v = dc.mm(hq.double(), wd.double().T) * (hs.double()[:, None] * sd.double()[None, :])
    bound = (dc.mm(near.double(), wd.double().abs().T) * hs.double()[:, None] + dc.mm(hq.double().abs(), wd.double().abs().T)
             * es[:, None]) * sd.double()[None, :] + v.abs() * (4 * dc.U32 + dc.half_ulp(f.t)) * 1.01 + dc.tiny(f.t)
    dc.check(y, (v, bound), "y")


def test_int_block_keeps_non_finite_rows_apart():
    f, codes, d = _int_block(6, 128, 64, "bf16")
    y = _run_int_block(f, codes, d)
    f.x[2, 7] = float("inf")
    f.x[4] = 0
    y2 = _run_int_block(f, codes, d)
    assert bool(torch.isnan(y2[2]).all()) and bool((y2[4] == 0).all())
    assert torch.equal(y[[0, 1, 3, 5]], y2[[0, 1, 3, 5]])


# ---------------------------------------------------------------- as a program makes them
def test_block_in_both_widths():
    """A run of the operators as they are used: the 16-bit block with its gradients, its weights quantised by the
    operator itself, and the 8-bit block and product on the same tokens, which stay near the 16-bit results."""
    f = dc.Ffn(48, 512, 256)
    y, gu = f.forward()
    dx = f.backward(gu)[0]
    assert bool(torch.isfinite(dx).all())
    codes = []
    for m in (f.wg, f.wu, f.wd):
        q, s = torch.empty(m.shape, dtype=torch.int8, device="cuda"), torch.empty(m.shape[0], device="cuda")
        ft.ft_moe_int_quantize(f.dt, *m.shape, m, q, s)
        codes += [q, s]
    d = ft.make_gated_ffn(f.dt, f.T, f.H, f.I)
    y8 = _run_int_block(f, codes, d)
    # 8-bit rows: a code is off by at most half a step of amax / 127; for normal rows amax < 5 sigma, a relative
    # 2-norm error of at most 5 / 127 / sqrt(12) per operand; five quantised operands (x, Wg, Wu, h, Wd), h with a
    # wider tail (amax < 25 sigma)
    step = 5 / 127 / 12**0.5
    far = (y8.double() - y.double()).norm() / y.double().norm()
    assert far <= (4 * step + 5 * step) * 1.5
    xq, xs = torch.empty(f.T, f.H, dtype=torch.int8, device="cuda"), torch.empty(f.T, device="cuda")
    ft.ft_moe_int_quantize(f.dt, f.T, f.H, f.x, xq, xs)
    g8 = torch.empty(f.T, f.I, device="cuda")
    m = ft.make_int_matmul(f.T, f.H, f.I, ft.FT_DT_F32)
    ft.ft_moe_int_matmul(m, xq, xs, codes[0], codes[1], g8, torch.empty(ft.ft_moe_int_matmul_work(m), dtype=torch.uint8, device="cuda"))
    dc.check(g8, dc.int_product_reference(xq, xs, codes[0], codes[1], torch.float32), "g")


def test_calls_on_a_stream():
    f = dc.Ffn(40, 256, 128)
    y, gu = f.forward()
    grads = f.backward(gu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2, gu2 = f.forward(stream=s)
    assert torch.equal(y, y2) and torch.equal(gu, gu2)
    assert all(torch.equal(a, b) for a, b in zip(f.backward(gu, stream=s), grads))


@pytest.mark.parametrize("T", [1, 24, 200])
def test_graph_replays(T):
    """Forward, backward and the 8-bit block captured into one graph: every replay, with eager work between, gives the
    eager bits for the inputs of that replay."""
    f, codes, d = _int_block(T, 512, 256, "bf16")
    w1, w2, w3 = f.work(False), f.work(True), torch.empty(ft.ft_moe_int_gated_ffn_work(d), dtype=torch.uint8, device="cuda")
    new = lambda r, c: torch.empty(r, c, dtype=f.t, device="cuda")  # noqa: E731
    y, gu, y8, dx = new(T, 512), new(T, 512), new(T, 512), new(T, 512)
    dwg, dwu, dwd = new(256, 512), new(256, 512), new(512, 256)

    def calls(stream):
        ft.ft_moe_gated_ffn_forward(f.desc, f.x, f.wg, f.wu, f.wd, y, gu, w1, stream)
        ft.ft_moe_gated_ffn_backward(f.desc, f.x, f.wg, f.wu, f.wd, gu, f.dy, dx, dwg, dwu, dwd, w2, stream)
        ft.ft_moe_int_gated_ffn(d, f.x, *codes, y8, w3, stream)

    outs = (y, gu, y8, dx, dwg, dwu, dwd)
    s = torch.cuda.Stream()
    calls(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls(torch.cuda.current_stream())
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for _ in range(4):
        f.x.copy_(torch.randn(T, 512, generator=g, device="cuda").to(f.t))
        calls(None)
        torch.cuda.synchronize()
        want = [v.clone() for v in outs]
        for v in outs:
            v.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_same_call_twice_gives_the_same_bits():
    f = dc.Ffn(77, 2048, 768)
    y, gu = f.forward()
    first = f.backward(gu)
    for _ in range(3):
        y2, gu2 = f.forward()
        assert torch.equal(y, y2) and torch.equal(gu, gu2)
        assert all(torch.equal(a, b) for a, b in zip(f.backward(gu), first))


def test_host_memory_is_refused():
    f = dc.Ffn(4, 32, 16)
    y = torch.empty(4, 32, dtype=f.t)  # host memory
    with pytest.raises(ft.FtError) as e:
        ft.ft_moe_gated_ffn_forward(f.desc, f.x, f.wg, f.wu, f.wd, y, None, f.work(False))
    assert e.value.code == ft.FT_E_INVALID and "y" in str(e.value)
    with pytest.raises(ft.FtError):
        ft.ft_moe_gated_ffn_forward(f.desc, f.x, f.wg.cpu(), f.wu, f.wd, torch.empty_like(f.x), None, f.work(False))


def test_gradients_of_frozen_or_first_blocks():
    """Nothing asked for is nothing done."""
    f = dc.Ffn(4, 32, 16)
    assert ft.ft_moe_gated_ffn_backward(f.desc, None, f.wg, f.wu, f.wd, f.saved(), f.dy) == ft.FT_OK


@pytest.mark.parametrize("type_", ["bf16", "fp16"])
@pytest.mark.parametrize("H,I", [(1024, 768), (136, 1000), (2048, 96), (45, 23), (1, 1)])
def test_int_block_rows_do_not_depend_on_their_number(H, I, type_):
    """Few tokens are quantised by the products themselves, more by launches of their own: the sums are exact and the
    codes correctly rounded, so a token's result has the same bits in either."""
    f, codes, d = _int_block(40, H, I, type_)
    f.x[1] = 0
    f.x[2] *= 2.0**-14
    f.x[5, H // 2] = float("nan")
    y = _run_int_block(f, codes, d)
    assert bool(y[5].isnan().all()) and bool((y[1] == 0).all())
    x = f.x
    for T in (1, 2, 3, 6, 8, 13, 16):
        for first in (0, 7):
            f.T, f.x = T, x[first:first + T]
            some = ft.make_gated_ffn(f.dt, T, H, I, ld_w_in=d.ld_w_in, ld_w_out=d.ld_w_out)
            got = _run_int_block(f, codes, some)
            assert torch.equal(got.view(torch.int16), y[first:first + T].view(torch.int16)), (T, first)


@pytest.mark.parametrize("size", [(4096, 2048, 768), (2049, 1024, 2048), (1500, 1000, 1016), (1300, 777, 901), (300, 512, 256)])
def test_gradients_do_not_depend_on_which_are_asked_for(size):
    """dx and the weight gradients may share a launch: the same bits as each alone, and again at each call."""
    f = dc.Ffn(*size, "fp16")
    gu = f.saved()
    work = f.work(True)
    both = f.backward(gu, work=work)
    dx = f.backward(gu, want_dw=False, work=work)[0]
    dw = f.backward(gu, want_dx=False, work=work)[1:]
    assert all(torch.equal(a, b) for a, b in zip((dx, *dw), both))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(f.backward(gu, work=work), both))


def test_gradients_with_the_same_tensor_twice():
    """x and dy in one buffer, and one matrix for both gates, are inputs like any others."""
    f = dc.Ffn(37, 45, 45)
    gu = f.saved()
    f.dy, f.wu = f.x, f.wg
    for want in (dict(), dict(want_dw=False), dict(want_dx=False)):
        got, ref = f.backward(gu, **want), f.backward_reference(gu)
        if want.get("want_dx", True):
            dc.check(got[0], ref[0], "dx")
        if want.get("want_dw", True):
            for g, r in zip(got[1:], ref[1:]):
                dc.check(g, r)


def test_two_streams_at_once():
    """Calls on two streams, each with scratch memory of its own, do not disturb each other."""
    fs = [dc.Ffn(1200, 1024, 512, seed=i) for i in range(2)]
    gus = [f.saved() for f in fs]
    want = [(f.forward()[0], *f.backward(gu)) for f, gu in zip(fs, gus)]
    streams, works = [torch.cuda.Stream() for _ in fs], [(f.work(False), f.work(True)) for f in fs]
    outs = []
    torch.cuda.synchronize()
    for _ in range(6):
        for f, gu, s, (w1, w2) in zip(fs, gus, streams, works):
            o = [torch.empty_like(v) for v in want[0]]
            torch.cuda.current_stream().synchronize()
            ft.ft_moe_gated_ffn_forward(f.desc, f.x, f.wg, f.wu, f.wd, o[0], None, w1, s)
            ft.ft_moe_gated_ffn_backward(f.desc, f.x, f.wg, f.wu, f.wd, gu, f.dy, *o[1:], w2, s)
            outs.append(o)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert all(torch.equal(a, b) for a, b in zip(o, want[i % 2]))


@pytest.mark.parametrize("off", [1, 3])
def test_addresses_off_the_grid(off):
    """Base addresses that are no multiples of 16 bytes, alone or with widths that are none either."""
    for T, H, I in ((3, 64, 48), (70, 64, 48), (70, 61, 43)):
        f = dc.Ffn(T, H, I)
        for name in ("x", "wg", "wd", "dy"):
            g = dc.Ffn(T, H, I)
            m = getattr(g, name)
            flat = torch.empty(m.numel() + 16, dtype=m.dtype, device="cuda")
            moved = flat[off:off + m.numel()].view(m.shape)
            moved.copy_(m)
            setattr(g, name, moved)
            y, gu = g.forward()
            (ry, rgu) = g.forward_reference()
            dc.check(y, ry, "y")
            dc.check(gu, rgu, "gu")
            for a, r in zip(g.backward(gu), g.backward_reference(gu)):
                dc.check(a, r, name)


@pytest.mark.parametrize("T", [2, 70])
def test_offsets_past_32_bits(T):
    """A weight matrix of more than 4 GB, and rows of tokens and results whose distances pass 4 GB together: the last
    rows and columns."""
    K, N, far = 8192, 600_000, 2000
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=g, device="cuda") + 0.5
    x = torch.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(T, generator=g, device="cuda") + 0.5
    y = torch.empty(T, N, device="cuda")
    d = ft.make_int_matmul(T, K, N, ft.FT_DT_F32)
    ft.ft_moe_int_matmul(d, x, xs, w, ws, y, torch.empty(ft.ft_moe_int_matmul_work(d), dtype=torch.uint8, device="cuda"))
    for part in (slice(0, far), slice(N - far, N)):
        dc.check(y[:, part], dc.int_product_reference(x, xs, w[part], ws[part], torch.float32), "y")
    del w, y
    step = (1 << 31) // T // 64 * 64 + 64  # elements: T rows of results pass 8 GB
    xw = torch.empty(T * step, dtype=torch.int8, device="cuda").view(T, step)[:, :K]
    xw.copy_(x)
    w = torch.randint(-128, 128, (far, K), generator=g, device="cuda", dtype=torch.int8)
    yw = torch.empty(T * step, dtype=torch.float32, device="cuda").view(T, step)[:, :far]
    d = ft.make_int_matmul(T, K, far, ft.FT_DT_F32, ld_x=step, ld_y=step)
    ft.ft_moe_int_matmul(d, xw, xs, w, ws, yw, torch.empty(ft.ft_moe_int_matmul_work(d), dtype=torch.uint8, device="cuda"))
    dc.check(yw, dc.int_product_reference(x, xs, w, ws[:far], torch.float32), "y")


@pytest.mark.parametrize("size", [(4096, 2048, 768), (1300, 777, 901)])
def test_backward_graph_replays(size):
    """A captured backward pass whose gradients share a launch (its work queue is cleared in the graph), and one whose
    operands are copied first: every replay, with eager calls on the same scratch memory between, gives the eager bits."""
    f = dc.Ffn(*size)
    T, H, I = size
    gu, work, s = f.saved(), f.work(True), torch.cuda.Stream()
    outs = [torch.empty(T, H, dtype=f.t, device="cuda"), *(torch.empty(I, H, dtype=f.t, device="cuda") for _ in range(2)),
            torch.empty(H, I, dtype=f.t, device="cuda")]

    def call(stream):
        ft.ft_moe_gated_ffn_backward(f.desc, f.x, f.wg, f.wu, f.wd, gu, f.dy, *outs, work, stream)

    torch.cuda.synchronize()
    call(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(torch.cuda.current_stream())
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for _ in range(4):
        f.dy.copy_(torch.randn(T, H, generator=g, device="cuda").to(f.t))
        call(None)
        torch.cuda.synchronize()
        want = [v.clone() for v in outs]
        for v in outs:
            v.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
