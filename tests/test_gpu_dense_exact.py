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
