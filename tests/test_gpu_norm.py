"""The norm with the residual's addition on the GPU against 64-bit references: rows, codes and gradients, over lengths,
odd sizes, strides and types; then the calls as a program makes them."""

import pytest
import torch

import lru_expert_cache_amd as ft
from tests import around_case as ac

pytestmark = pytest.mark.gpu

# (rows, cols, row padding)
SIZES = [
    (1, 1, 0), (3, 7, 0), (2, 8, 0), (5, 9, 1), (1, 64, 0), (4, 100, 3), (1, 2048, 0), (2, 511, 0), (3, 512, 8),
    (7, 513, 0), (33, 1000, 24), (2, 2047, 1), (9, 2049, 0), (32, 6144, 0), (5, 4097, 7), (65, 7168, 64), (3, 8191, 0),
    (2, 8193, 0), (3, 16384, 0), (2, 20001, 3), (2, 32768, 0), (2, 32769, 0), (1, 70000, 0), (1500, 256, 0), (1031, 2050, 6),
]
TYPES = [("bf16", None), ("fp16", None), ("fp32", None), ("bf16", "fp32"), ("fp16", "fp32")]


def _check_forward(n, got, ref, codes=True):
    ac.check(got["sum"], ref["sum"], "sum")
    ac.check(got["y"], ref["y"], "y")
    if codes:
        assert torch.equal(got["scale"], ref["scale"])
        assert torch.equal(got["codes"], ref["codes"]), int((got["codes"] != ref["codes"]).sum())


@pytest.mark.parametrize("type_,res", TYPES)
@pytest.mark.parametrize("size", SIZES)
def test_forward(size, type_, res):
    n = ac.Norm(*size[:2], type_, res, size[2])
    got, ref = n.forward(), n.forward_reference()
    _check_forward(n, got, ref)
    # each output alone has the same bits, without a residual too
    assert torch.equal(n.forward(sum_=False, codes=False)["y"], got["y"])
    alone = n.forward(sum_=False, y=False)
    assert torch.equal(alone["codes"], got["codes"]) and torch.equal(alone["scale"], got["scale"])
    assert torch.equal(n.forward(y=False, codes=False)["sum"], got["sum"])
    _check_forward(n, n.forward(residual=False), n.forward_reference(residual=False))


@pytest.mark.parametrize("type_,res", TYPES)
@pytest.mark.parametrize("size", SIZES)
def test_backward(size, type_, res):
    n = ac.Norm(*size[:2], type_, res, size[2])
    got, ref = n.backward(), n.backward_reference()
    for k, v in ref.items():
        ac.check(got[k], v, k)
    assert torch.equal(n.backward(dresidual=False, dweight=False)["dx"], got["dx"])
    assert torch.equal(n.backward(dx=False, dweight=False)["dresidual"], got["dresidual"])
    assert torch.equal(n.backward(dx=False, dresidual=False)["dweight"], got["dweight"])
    got, ref = n.backward(dsum=False), n.backward_reference(dsum=False)
    for k, v in ref.items():
        ac.check(got[k], v, k)


def test_codes_are_those_of_the_row_quantiser():
    """Rows that the norm leaves as they are (fp32, mean square 1, weight 1, eps 0): ft_moe_int_quantize's codes."""
    g = ac.gen(3)
    x = torch.where(torch.rand(40, 512, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    d = ft.make_rms_norm(ft.FT_DT_F32, 40, 512, 0.0)
    w = torch.rand(512, generator=g, device="cuda")
    y, codes, scale = torch.empty_like(x), torch.empty(40, 512, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
    ft.ft_moe_rms_norm_forward(d, x, None, w, None, y, codes, scale)
    c2, s2 = torch.empty_like(codes), torch.empty_like(scale)
    ft.ft_moe_int_quantize(ft.FT_DT_F32, 40, 512, y, c2, s2)
    assert torch.equal(y, x * w) and torch.equal(codes, c2) and torch.equal(scale, s2)


def test_rows_of_zeros_infinities_and_nan():
    for cols in (5, 64, 2048, 40000):
        n = ac.Norm(6, cols)
        before = n.forward()
        n.x[1], n.residual[1] = 0, 0
        n.x[2, cols // 2] = float("inf")
        n.x[3, cols - 1] = float("nan")
        n.x[4, 0], n.residual[4, 0] = float("inf"), float("-inf")
        got = n.forward()
        assert (got["y"][1] == 0).all() and (got["codes"][1] == 0).all() and got["scale"][1] == 0
        for r in (2, 3, 4):
            assert torch.isnan(got["scale"][r]) and (got["codes"][r] == 0).all()
        assert torch.isnan(got["y"][2, cols // 2]) and (cols == 1 or (got["y"][2, 0] == 0))
        assert torch.isnan(got["y"][3]).all() and torch.isnan(got["y"][4]).all()
        for r in (0, 5):
            for k in got:
                assert torch.equal(got[k][r], before[k][r])
        # an infinite weight leaves an infinity in every row
        n.weight[cols - 1] = float("inf")
        got = n.forward()
        assert torch.isnan(got["scale"]).all() and (got["codes"] == 0).all()


def test_extreme_magnitudes():
    """Squares and quotients beyond the range of 32 bits."""
    g = ac.gen(5)
    for scale in (1e30, 1e-30, 1e-38, 2.0**-140):
        n = ac.Norm(5, 600, "fp32", eps=0.0)
        n.x.copy_(torch.randn(5, 600, generator=g, device="cuda") * scale)
        n.residual.zero_()
        got, ref = n.forward(), n.forward_reference()
        _check_forward(n, got, ref)
    # small results: scales among the smallest numbers
    n = ac.Norm(3, 300, "fp32", eps=1.0)
    n.residual.zero_()
    for scale in (2.0**-125, 2.0**-142, 2.0**-149):
        n.x.copy_((torch.randn(3, 300, generator=g, device="cuda") * scale * 8))
        _check_forward(n, n.forward(), n.forward_reference())
    n = ac.Norm(4, 600, "fp32", eps=0.0)
    for scale in (1e25, 1e-25):
        n.s.copy_(torch.randn(4, 600, generator=g, device="cuda") * scale)
        n.dsum.copy_(torch.randn(4, 600, generator=g, device="cuda") / scale)
        got, ref = n.backward(), n.backward_reference()
        for k, v in ref.items():
            ac.check(got[k], v, k)


def test_gradients_follow_differences():
    n = ac.Norm(5, 40, "fp32", seed=2)
    got, ref = n.backward(), n.backward_reference()
    g = ac.gen(6)

    def loss(s, w):
        return (s / torch.sqrt((s * s).mean(1, keepdim=True) + n.eps) * w * n.dy.double()).sum() + (s * n.dsum.double()).sum()

    at = [n.s.double(), n.weight.double()]
    for i, k in enumerate(("dx", "dweight")):
        v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 2.0**-14
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + step * v, at[i] - step * v
        difference = (loss(*hi) - loss(*lo)) / (2 * step)
        # a central difference is off by step^2 / 6 of the third derivative: 2^-28 / 6 of values of the gradient's order
        # (s of size 2: each derivative divides by about s, and has a few terms)
        bound = (ref[k][1] * v.abs()).sum() + 1e-6 * (ref[k][0] * v).abs().sum()
        assert (difference - (got[k].double() * v).sum()).abs() <= bound


@pytest.mark.parametrize("cols", [96, 40000])
def test_in_place(cols):
    n = ac.Norm(9, cols, "bf16", pad=8)
    ref = n.forward()
    x, residual = n.x.clone(), n.residual.clone()
    for target in ("residual", "x"):
        # views of the padded buffers keep their row distance
        n.x.copy_(x)
        n.residual.copy_(residual)
        out = getattr(n, target)
        other = n.x if target == "residual" else n.residual
        ft.ft_moe_rms_norm_forward(n.d, n.x, n.residual, n.weight, out, other)
        assert torch.equal(out, ref["sum"]) and torch.equal(other, ref["y"])
    ref = n.backward()
    for dx, dres in (("dy", "dsum"), ("dsum", "s"), ("s", "dy")):
        m = ac.Norm(9, cols, "bf16", pad=8)
        dw = torch.empty(cols, dtype=m.t, device="cuda")
        ft.ft_moe_rms_norm_backward(m.d, m.s, m.weight, m.dy, m.dsum, getattr(m, dx), getattr(m, dres), dw, m.work())
        assert torch.equal(getattr(m, dx), ref["dx"]) and torch.equal(getattr(m, dres), ref["dresidual"])
        assert torch.equal(dw, ref["dweight"])


def test_no_rows():
    n = ac.Norm(0, 130, "fp16")
    n.forward()
    assert (n.backward()["dweight"] == 0).all()


def test_rows_at_odd_addresses():
    """Rows off every grid but the elements' own."""
    buf = torch.randn(40 * 1001 + 64, device="cuda").to(torch.bfloat16)
    for off in (1, 3, 7):
        x, res = buf[off:off + 20 * 1001].view(20, 1001), buf[20 * 1001 + off + 2:][:20 * 1001].view(20, 1001)
        n = ac.Norm(20, 1001)
        n.d.ld_x = n.d.ld_residual = 1001
        n.x, n.residual = x, res
        got, ref = n.forward(), n.forward_reference()
        _check_forward(n, got, ref)


@pytest.mark.parametrize("cols", [3, 8])
def test_millions_of_rows(cols):
    n = ac.Norm((1 << 21) + 3, cols)
    got, ref = n.forward(), n.forward_reference()
    _check_forward(n, got, ref)
    got, ref = n.backward(), n.backward_reference()
    for k, v in ref.items():
        ac.check(got[k], v, k)


def test_rows_beyond_4_gb():
    """Offsets of more than 32 bits: rows far apart."""
    n = ac.Norm(40, 300)
    fwd, bwd, ld = n.forward(), n.backward(), 1 << 26
    far = lambda v: torch.as_strided(torch.empty(39 * ld + 300, dtype=v.dtype, device="cuda"), (40, 300), (ld, 1)).copy_(v)  # noqa: E731
    assert 39 * ld * 2 > 2**32
    y = far(n.x)
    n.d.ld_x = n.d.ld_y = n.d.ld_residual = n.d.ld_sum = n.d.ld_codes = ld
    x, res = far(n.x), far(n.residual)
    codes, scale = far(fwd["codes"] * 0), torch.empty(40, device="cuda")
    ft.ft_moe_rms_norm_forward(n.d, x, res, n.weight, res, y, codes, scale)
    assert torch.equal(res, fwd["sum"]) and torch.equal(y, fwd["y"]) and torch.equal(codes, fwd["codes"])
    s, dy, dsum = far(n.s), far(n.dy), far(n.dsum)
    ft.ft_moe_rms_norm_backward(n.d, s, n.weight, dy, dsum, dy, dsum, None, n.work())
    assert torch.equal(dy, bwd["dx"]) and torch.equal(dsum, bwd["dresidual"])


@pytest.mark.parametrize("cols", [5, 8, 12, 100, 512, 1000, 2050, 7168, 16383, 20001])
def test_infinite_gradients(cols):
    """An infinity in dy, wherever it stands in its row: infinities and NaN where the formula has them."""
    at = sorted({0, cols // 2, max(0, cols - 9), cols - 8 if cols >= 8 else 0, cols - 1})
    n = ac.Norm(len(at) + 1, cols, "bf16", "fp32", pad=3)
    before = n.backward()
    for row, c in enumerate(at):
        n.dy[row, c] = float("inf") if row % 2 else float("-inf")
    got, ref = n.backward(), n.backward_reference()
    for k in ("dx", "dresidual"):
        want = ref[k][0][:-1]
        assert torch.equal(torch.isnan(got[k][:-1]), torch.isnan(want)), k
        assert torch.equal(got[k][:-1].double() == torch.inf, want == torch.inf), k
        assert torch.equal(got[k][:-1].double() == -torch.inf, want == -torch.inf), k
        assert torch.equal(got[k][-1], before[k][-1])
    inf = torch.zeros(cols, dtype=torch.bool, device="cuda")
    inf[at] = True
    assert torch.equal(~torch.isfinite(got["dweight"]), inf)


@pytest.mark.parametrize("type_,res", [("fp32", None), ("bf16", "fp32"), ("bf16", None)])
@pytest.mark.parametrize("cols", [5, 600, 7168, 16400])
def test_gradients_of_the_smallest_and_largest_rows(cols, type_, res):
    """1 / sqrt(mean(s^2)) beyond the range of 32 bits, either way, with gradients that are within it."""
    g = ac.gen(9)
    for size, dy in ((2.0**-130, 2.0**-20), (2.0**-145, 2.0**-60), (2.0**-110, 1.0), (2.0**110, 2.0**60), (2.0**125, 2.0**60)):
        n = ac.Norm(4, cols, type_, res, pad=1, eps=0.0)
        if size < 2.0**-133 and n.r == torch.bfloat16:
            continue  # below the type's smallest number
        n.s.copy_((torch.rand(4, cols, generator=g, device="cuda") - 0.5) * size)
        n.dy.copy_(torch.randn(4, cols, generator=g, device="cuda") * dy)
        n.dsum.zero_()
        assert (n.s != 0).any(1).all() and torch.isfinite(n.s).all()
        got, ref = n.backward(), n.backward_reference()
        for k, v in ref.items():
            assert torch.isfinite(v[0]).all() and v[0].abs().max() < 2.0**127
            ac.check(got[k], v, f"{k} {size}")


def test_gradients_without_scratch_memory():
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    for rows, cols in ((1, 8), (2, 2050), (2, 16384)):
        n = ac.Norm(rows, cols, "bf16", "fp32", pad=1)
        got, ref = n.backward(work=none), n.backward_reference()
        for k, v in ref.items():
            ac.check(got[k], v, k)
    for rows, cols in ((70, 2050), (3, 9)):
        n = ac.Norm(rows, cols, "fp16", pad=1)
        want, got = n.backward(), n.backward(dweight=False, work=none)
        assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dresidual"], want["dresidual"])
    # rows that no workgroup holds: what a call without the weight's gradient uses is less than one with it is told
    n = ac.Norm(5, 20001, "bf16")
    want, got = n.backward(), n.backward(dweight=False, work=torch.empty(5 * 16 + 176, dtype=torch.uint8, device="cuda"))
    assert torch.equal(got["dx"], want["dx"])


@pytest.mark.parametrize("type_,res", TYPES)
def test_rows_are_rounded_by_way_of_32_bits(type_, res):
    """The sum, bit for bit: exact in 64 bits for 16-bit addends and rounded once to 32, then once to its type."""
    n = ac.Norm(50, 1500, type_, res, seed=4)
    s = (n.x.double() + n.residual.double()).float()
    assert torch.equal(n.forward()["sum"], s.to(n.r))
