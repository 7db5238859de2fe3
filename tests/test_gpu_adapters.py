"""Low-rank adapters on the GPU against 64-bit references: lengths, odd sizes, strides, types and orders of ids."""

import pytest
import torch

import lru_expert_cache_amd as ft
from tests import around_case as ac

pytestmark = pytest.mark.gpu

# (tokens, in, out, rank, adapters, row padding of tokens, of weights)
SIZES = [
    (1, 1, 1, 1, 1, 0, 0), (1, 64, 64, 8, 1, 0, 0), (2, 33, 17, 3, 2, 0, 0), (5, 100, 70, 5, 9, 3, 1),
    (1, 2048, 2048, 16, 8, 0, 0), (16, 256, 520, 16, 4, 8, 8), (17, 255, 129, 12, 3, 0, 5), (32, 6144, 1024, 16, 32, 0, 0),
    (33, 1000, 777, 24, 40, 1, 0), (64, 512, 96, 32, 5, 0, 0), (65, 640, 300, 64, 2, 0, 0), (70, 2050, 31, 17, 100, 0, 0),
    (100, 96, 2048, 33, 7, 64, 8), (257, 384, 640, 128, 3, 0, 0), (130, 130, 130, 256, 2, 2, 2), (300, 72, 1032, 100, 6, 0, 0),
    (777, 320, 200, 8, 48, 0, 0), (1531, 2048, 503, 8, 48, 64, 0), (2500, 128, 264, 16, 1, 0, 0),
]
FORMS = [("bf16", "same", None), ("fp16", "same", None), ("bf16", "fp32", None), ("fp16", "fp32", "fp32"), ("bf16", "fp32", "fp32"),
         ("fp16", "fp32", None), ("bf16", None, None), ("fp16", None, "fp32")]


@pytest.mark.parametrize("type_,base,out", FORMS)
@pytest.mark.parametrize("size", SIZES)
def test_apply(size, type_, base, out):
    T, K, N, R, n, pad, wpad = size
    c = ac.Adapters(T, K, N, R, n, type_, base, out, pad, wpad)
    y = c.apply()
    ac.check(y, c.reference(), "y")
    assert torch.equal(y, c.apply())


@pytest.mark.parametrize("type_,base,out", FORMS)
@pytest.mark.parametrize("in_", [7, 63, 200, 1000, 2048, 2560, 2561, 5000])
def test_few_tokens(in_, type_, base, out):
    """One launch, or two, for the same tokens: widths on either side, ranks on either side of a piece of eight."""
    for tokens, N, R, n in ((1, 2100, 16, 3), (9, 65, 7, 4), (37, 1030, 13, 2), (64, 300, 8, 64)):
        c = ac.Adapters(tokens, in_, N, R, n, type_, base, out, pad=1, seed=in_)
        ac.check(c.apply(), c.reference(), f"{tokens} tokens")


@pytest.mark.parametrize("type_,base,out", FORMS)
@pytest.mark.parametrize("tokens,in_,N", [(64, 72, 20001), (50, 72, 8200), (64, 2600, 20001)])
def test_few_tokens_into_many_columns(tokens, in_, N, type_, base, out):
    """A workgroup takes several steps of columns."""
    c = ac.Adapters(tokens, in_, N, 16, 64, type_, base, out, ids=[(7 * i) % 64 for i in range(tokens)])
    ac.check(c.apply(), c.reference())


@pytest.mark.parametrize("tokens", [7, 64, 90, 1200, 9000])
@pytest.mark.parametrize("order", ["one", "none", "runs", "all", "reverse", "far"])
def test_orders(tokens, order):
    n = 70
    i = torch.arange(tokens)
    ids = {"one": torch.full((tokens,), 3), "none": torch.full((tokens,), -1), "runs": (i // 23) % n, "all": i % n,
           "reverse": (tokens - 1 - i) * n // tokens, "far": torch.where(i % 3 == 0, i % n, torch.where(i % 3 == 1, n + i, -(2**31) + i))}[order]
    c = ac.Adapters(tokens, 136, 200, 16, n, ids=ids)
    ac.check(c.apply(), c.reference(), order)


def test_tokens_do_not_depend_on_each_other():
    """The same token gives the same bits wherever it stands, and a NaN stays in its row."""
    c = ac.Adapters(150, 512, 384, 16, 5)
    y = c.apply()
    perm = torch.randperm(150, device="cuda")
    c.x, c.base = c.x[perm].contiguous(), c.base[perm].contiguous()
    c.ids = c.ids[perm].contiguous()
    assert torch.equal(c.apply(), y[perm])
    c.x[40, 100], c.ids[40] = float("nan"), 2
    c.x[41, 100], c.ids[41] = float("inf"), -1
    c.x[42, 100], c.ids[42] = float("inf"), 1
    z = c.apply()
    keep = torch.ones(150, dtype=torch.bool, device="cuda")
    keep[40:43] = False
    assert torch.equal(z[keep], y[perm][keep])
    assert torch.isnan(z[40]).all() and torch.equal(z[41], c.base[41].to(z.dtype)) and not torch.isfinite(z[42]).any()


def test_weights_of_other_adapters_are_not_read():
    c = ac.Adapters(60, 256, 130, 16, 6)
    c.ids = torch.where(c.ids >= 4, 1, c.ids)
    y = c.apply()
    c.a[4 * 16:], c.b[4 * 130:] = float("nan"), float("nan")
    assert torch.equal(c.apply(), y)


@pytest.mark.parametrize("x,a,scale", [(900.0, 85.0, 2.0**-22), (2.0**-12, 2.0**-13, 2.0**22)])
def test_sums_beyond_fp16s_range(x, a, scale):
    """A x of millions, or of 2^-20 and less: results of the order of 1."""
    c = ac.Adapters(40, 512, 96, 16, 3, "fp16", None)
    for v, size in ((c.x, x), (c.a, a)):
        v.copy_(v.float() / v.float().std() * size)
        assert torch.isfinite(v).all()
    c.scale = torch.full((3,), scale, device="cuda")
    h = c.x.float().abs().mean() * c.a.float().abs().mean() * 512**0.5
    assert h > 2.0**17 or h < 2.0**-18
    ac.check(c.apply(), c.reference())


@pytest.mark.parametrize("type_,base,out", FORMS)
@pytest.mark.parametrize("size", [(8500, 4200, 4100, 40, 3), (4100, 6000, 2203, 5, 2), (4096, 4104, 4096, 64, 20), (2100, 520, 1030, 100, 3),
                                  (1030, 70, 260, 128, 2), (3000, 300, 260, 30, 5)])
def test_large_tiles(size, type_, base, out):
    """Tiles of 64 and 32 tokens, several windows, odd widths."""
    c = ac.Adapters(*size, type_, base, out)
    c.ids = torch.sort(c.ids).values.contiguous()  # long runs
    ac.check(c.apply(), c.reference(), "y")


def test_more_work_than_a_launch_has_workgroups():
    """Many windows, each with room for thousands of adapters: workgroups go round; rows picked from all over."""
    T, N, n = 300_000, 51_200, 4096
    g = ac.gen(1)
    x, a = torch.randn(T, 8, generator=g, device="cuda").to(torch.bfloat16), torch.randn(n, 1, 8, generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randn(n, N, 1, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    d = ft.make_adapters(ft.FT_DT_BF16, T, 8, N, 1, n)
    ft.ft_moe_adapters_apply(d, x, ids, a, b, None, None, y, torch.empty(ft.ft_moe_adapters_work(d), dtype=torch.uint8, device="cuda"))
    at = torch.cat([torch.tensor([0, 1, 8191, 8192, T - 1], device="cuda"), torch.randint(0, T, (60,), generator=g, device="cuda")])
    i = ids[at].long()
    h = (x[at].double() * a[i, 0].double()).sum(1)
    v = torch.where((i >= 0)[:, None], h[:, None] * b[i, :, 0].double(), 0.0)
    hm = (x[at].double() * a[i, 0].double()).abs().sum(1)[:, None] * b[i, :, 0].double().abs()
    ac.check(y[at], (v, ac.rounded(v, y.dtype, hm * (10 * 2 * ac.E + 2.0**-17 + 14 * ac.E))), "y")


@pytest.mark.parametrize("T", [40, 90, 5000])
def test_in_place(T):
    c = ac.Adapters(T, 256, 300, 16, 4, pad=8)
    y, before = c.apply(), c.base.clone()
    ft.ft_moe_adapters_apply(c.d, c.x, c.ids, c.a, c.b, c.scale, c.base, c.base, c.work())
    assert torch.equal(c.base, y)
    none = c.ids < 0
    assert none.any() and torch.equal(c.base[none], before[none])


def test_without_scale_and_without_tokens():
    c = ac.Adapters(20, 64, 64, 8, 3, scale=False)
    ac.check(c.apply(), c.reference())
    ft.ft_moe_adapters_apply(ac.Adapters(0, 64, 64, 8, 3).d, None, None, None, None, None, None, None, None)


def _far(v, ld):
    """The same rows, ld elements apart."""
    t = torch.as_strided(torch.empty((v.shape[0] - 1) * ld + v.shape[1], dtype=v.dtype, device="cuda"), v.shape, (ld, 1))
    return t.copy_(v)


def test_rows_beyond_4_gb():
    """Offsets of more than 32 bits: matrices, tokens and results with their rows far apart."""
    c = ac.Adapters(50, 512, 600, 16, 40, ids=[39 - i % 3 for i in range(50)])
    y = c.apply()
    c.d.ld_a = 1 << 22
    c.a = _far(c.a, c.d.ld_a)
    assert torch.equal(c.apply(), y)
    c.d.ld_b = 1 << 17
    c.b = _far(c.b, c.d.ld_b)
    assert torch.equal(c.apply(), y)
    c.d.ld_x = c.d.ld_base = 1 << 26
    c.x, c.base = _far(c.x, c.d.ld_x), _far(c.base, c.d.ld_base)
    c.d.ld_y = 1 << 26
    out = _far(torch.zeros_like(y), c.d.ld_y)
    ft.ft_moe_adapters_apply(c.d, c.x, c.ids, c.a, c.b, c.scale, c.base, out, c.work())
    assert torch.equal(out, y)
