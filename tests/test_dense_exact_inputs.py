"""The inputs of the bit-for-bit tests of the dense operators, without a GPU: every sum is exact, and an oracle that
leaves out the last term along a K, as a kernel with a wrong remainder would, differs in most of its results (in at
least a fifth of any: a 16 x 16 fragment then shows it)."""

import pytest
import torch

from tests import dense_case as dc
from tests import dense_exact as de

SIZES = de.SMALL + de.TILED
SHOWS = 0.2


def shows(v, term, t):
    """The share of a sum's results that change, once rounded, when `term` is left out."""
    return float((v.to(t) != (v - term).to(t)).double().mean())


@pytest.mark.parametrize("size", SIZES)
def test_forward_inputs(size):
    T, H, I = size
    v = de.Values(*size).to("cpu", torch.float32)
    y, gu, h, sums = v.forward(torch.bfloat16)
    last = v.x[:, -1:] @ torch.cat([v.wg, v.wu], 0)[:, -1:].T
    assert shows(gu.float(), last, torch.bfloat16) == 1  # whole numbers up to 256: nothing hides
    for t in (torch.bfloat16, torch.float16):
        assert bool(torch.isfinite(sums.to(t)).all())
        assert shows(sums, h[:, -1:] @ v.wd[:, -1:].T, t) > SHOWS
        if T <= de.LO_FORWARD:  # and what a rounding of h would leave off
            assert shows(sums, sums - h.to(t).float() @ v.wd.T, t) > 0.05 or t == torch.float16


@pytest.mark.parametrize("size", SIZES)
def test_backward_inputs(size):
    v = de.Values(*size).to("cpu", torch.float32)
    dx, dwg, dwu, dwd, (dg, du, h) = v.backward(torch.bfloat16)
    some = slice(0, 64)
    sub = de.Values.__new__(de.Values)
    sub.I, sub.gu = min(64, v.I), torch.cat([v.gu[:, :v.I][:, some], v.gu[:, v.I:][:, some]], 1)
    _, less, _ = sub.dgu(v.dy[:, -1:] @ v.bd[-1:, some])  # what du lacks without the last term of dh
    for t in (torch.bfloat16, torch.float16):
        assert all(bool(torch.isfinite(m.to(t)).all()) for m in (dx, dwg, dwu, dwd))
        assert shows(dx, dg[:, -1:] @ v.bg[-1:], t) > SHOWS
        assert shows(dx, du[:, -1:] @ v.bu[-1:], t) > SHOWS
        assert shows(dwg, dg[-1:].T @ v.bx[-1:], t) > SHOWS
        assert shows(dwu, du[-1:].T @ v.bx[-1:], t) > SHOWS
        assert shows(dwd, v.dy[-1:].T @ h[-1:], t) > SHOWS * float((v.dy[-1] != 0).float().mean())
        assert shows(dwu[some], less.T @ v.bx, t) > SHOWS
        # and what a rounding of dg, du and h would leave off (one token has too few terms for it),
        if v.T <= de.LO_BACKWARD and t == torch.bfloat16:
            for m, rounded in ((dx, (dg.to(t).float() @ v.bg) + (du.to(t).float() @ v.bu)), (dwg, dg.to(t).float().T @ v.bx),
                               (dwu, du.to(t).float().T @ v.bx), (dwd, v.dy.T @ h.to(t).float()))[:0 if v.T == 1 else 4]:
                assert shows(m, m - rounded, t) > 0.01


@pytest.mark.parametrize("size", de.SMALL + de.TILED[:2])
def test_int_inputs(size):
    v = de.IntValues(*size).to("cpu", torch.float32)
    y, q, hs, sums = v.forward(torch.bfloat16)
    x, scale = dc.row_codes(v.x)
    assert torch.equal(x.float(), v.x) and bool((scale == 1).all())
    last = q[:, -1:].float() @ v.wd[:, -1:].T
    for t in (torch.bfloat16, torch.float16):
        y = (sums * hs[:, None] * v.down).to(t)
        assert bool(torch.isfinite(y).all())
        assert shows(sums, last, torch.float32) > SHOWS
    assert shows(v.x @ v.wu.T, v.x[:, -1:] @ v.wu[:, -1:].T, torch.bfloat16) == 1
