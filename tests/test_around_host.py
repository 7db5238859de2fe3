"""Norm, adapters and router balance without a GPU: refusals that come before
any device call, scratch sizes, and calls that have nothing to do."""

import ctypes

import pytest

import lru_expert_cache_amd as ft
from tests.test_dense_host import A, _Buf, _refused


def _norm(**kw):
    d = dict(dtype=ft.FT_DT_BF16, rows=4, cols=32, eps=1e-6)
    d.update(kw)
    return ft.make_rms_norm(**d)


def _adapters(**kw):
    d = dict(dtype=ft.FT_DT_BF16, tokens=4, in_features=32, out_features=48, rank=8, adapters=3)
    d.update(kw)
    return ft.make_adapters(**d)


def _balance(**kw):
    d = dict(dtype=ft.FT_DT_F32, tokens=4, experts=16, top_k=2, weight=0.01)
    d.update(kw)
    return ft.make_balance(**d)


def _forward(d, **kw):
    p = dict(x=A, residual=2 * A, weight=3 * A, sum=4 * A, y=5 * A, codes=6 * A, scale=7 * A)
    p.update(kw)
    return ft.ft_moe_rms_norm_forward(d, **p)


def _backward(d, **kw):
    p = dict(sum=A, weight=2 * A, dy=3 * A, dsum=4 * A, dx=5 * A, dresidual=6 * A, dweight=7 * A, work=_Buf(1 << 20))
    p.update(kw)
    return ft.ft_moe_rms_norm_backward(d, **p)


def _apply(d, **kw):
    p = dict(x=A, ids=2 * A, a=3 * A, b=4 * A, scale=5 * A, base=6 * A, y=7 * A, work=_Buf(1 << 20))
    p.update(kw)
    return ft.ft_moe_adapters_apply(d, **p)


def _balanced(d, **kw):
    p = dict(logits=A, valid=2 * A, sel=3 * A, w=4 * A, counts=5 * A, loss=6 * A, work=_Buf(1 << 20))
    p.update(kw)
    return ft.ft_moe_balance_forward(d, **p)


def _unbalanced(d, **kw):
    p = dict(logits=A, valid=2 * A, sel=3 * A, w=4 * A, counts=5 * A, dw=6 * A, dloss=7 * A, dlogits=8 * A)
    p.update(kw)
    return ft.ft_moe_balance_backward(d, **p)


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(dtype=4), dict(residual_dtype=ft.FT_DT_F16), dict(residual_dtype=-1),
                                dict(rows=-1), dict(rows=1 << 24), dict(cols=0), dict(cols=1 << 24), dict(eps=-1e-9),
                                dict(eps=float("nan")), dict(eps=float("inf")), dict(ld_x=31), dict(ld_residual=-1),
                                dict(ld_sum=8), dict(ld_y=1 << 32), dict(ld_codes=31)])
def test_bad_norms(kw):
    d = _norm(**kw)
    _refused(ft.ft_moe_rms_norm_work, d)
    _refused(_forward, d)
    _refused(_backward, d)


@pytest.mark.parametrize("kw", [dict(dtype=ft.FT_DT_F32), dict(dtype=0), dict(out_dtype=ft.FT_DT_F16), dict(base_dtype=ft.FT_DT_F16),
                                dict(out_dtype=ft.FT_DT_F32, base_dtype=ft.FT_DT_BF16), dict(tokens=-1), dict(tokens=1 << 24),
                                dict(in_features=0), dict(out_features=0), dict(rank=0), dict(rank=257), dict(adapters=0),
                                dict(adapters=4097), dict(ld_x=31), dict(ld_a=31), dict(ld_b=7), dict(ld_base=47),
                                dict(ld_y=1 << 32), dict(out_features=(1 << 24) - 1, adapters=4096, ld_b=(1 << 32) - 1)])
def test_bad_adapters(kw):
    d = _adapters(**kw)
    _refused(ft.ft_moe_adapters_work, d)
    _refused(_apply, d)


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(dtype=4), dict(tokens=-1), dict(tokens=1 << 24), dict(experts=0),
                                dict(experts=513), dict(top_k=0), dict(top_k=17), dict(experts=3, top_k=4),
                                dict(weight=float("inf")), dict(weight=float("nan")), dict(ld_logits=15)])
def test_bad_balances(kw):
    d = _balance(**kw)
    _refused(ft.ft_moe_balance_work, d)
    _refused(_balanced, d)
    _refused(_unbalanced, d)


def test_null_descriptions_and_sizes():
    L = ft.lib()
    n = ctypes.c_int64()
    for fn, d in ((L.ft_moe_rms_norm_work, _norm()), (L.ft_moe_adapters_work, _adapters()), (L.ft_moe_balance_work, _balance())):
        assert fn(None, ctypes.byref(n)) == ft.FT_E_INVALID
        assert fn(ctypes.byref(d), None) == ft.FT_E_INVALID


def test_missing_and_misaligned_pointers():
    for name in ("x", "weight"):
        _refused(_forward, _norm(), **{name: None})
    for name in ("x", "residual", "weight", "sum", "y"):
        _refused(_forward, _norm(), **{name: 9 * A + 1})
    _refused(_forward, _norm(), scale=9 * A + 2)
    _refused(_forward, _norm(residual_dtype=ft.FT_DT_F32), sum=9 * A + 2)
    _refused(_forward, _norm(), scale=None)  # codes without their scale
    _refused(_forward, _norm(), codes=None)
    for name in ("sum", "weight", "dy"):
        _refused(_backward, _norm(), **{name: None})
    for name in ("sum", "weight", "dy", "dsum", "dx", "dresidual", "dweight"):
        _refused(_backward, _norm(), **{name: 9 * A + 1})
    for name in ("x", "ids", "a", "b", "y"):
        _refused(_apply, _adapters(), **{name: None})
    for name in ("x", "ids", "a", "b", "scale", "base", "y"):
        _refused(_apply, _adapters(), **{name: 9 * A + 1})
    for name in ("logits", "sel", "w", "counts", "loss"):
        _refused(_balanced, _balance(), **{name: None})
        _refused(_balanced, _balance(), **{name: 9 * A + 1})
    for name in ("logits", "sel", "w", "counts", "dlogits"):
        _refused(_unbalanced, _balance(), **{name: None})
    for name in ("logits", "sel", "w", "counts", "dw", "dloss", "dlogits"):
        _refused(_unbalanced, _balance(), **{name: 9 * A + 1})


def test_scratch_memory_is_checked():
    for call, d, work in ((_backward, _norm(), ft.ft_moe_rms_norm_work), (_apply, _adapters(), ft.ft_moe_adapters_work),
                          (_balanced, _balance(), ft.ft_moe_balance_work)):
        n = work(d)
        assert n > 0
        _refused(call, d, work=_Buf(n - 1))
        _refused(call, d, work=None)
        _refused(call, d, work=_Buf(n, 64 * A + 8))  # not 16-byte aligned


def test_outputs_over_inputs():
    row = 32 * 2  # bytes of a norm's row
    _refused(_forward, _norm(), y=A + row)  # rows of x, one later
    _refused(_forward, _norm(ld_y=64), y=A)  # rows of x at another distance
    _refused(_forward, _norm(residual_dtype=ft.FT_DT_F32), sum=A)  # rows of x as another type
    _refused(_forward, _norm(), y=4 * A)  # sum
    _refused(_forward, _norm(), codes=A)
    _refused(_forward, _norm(), scale=3 * A)
    _refused(_forward, _norm(), sum=3 * A)  # weight
    _refused(_forward, _norm(), sum=3 * A - 4 * row + 2)
    _refused(_backward, _norm(), dx=2 * A)  # weight
    _refused(_backward, _norm(), dweight=3 * A)
    _refused(_backward, _norm(), dweight=5 * A)
    _refused(_backward, _norm(), dx=3 * A + row)
    _refused(_backward, _norm(), dx=6 * A)  # both outputs in one place
    _refused(_backward, _norm(), work=_Buf(1 << 20, 3 * A))
    _refused(_apply, _adapters(), y=A)
    for at in range(1, 6):
        _refused(_apply, _adapters(), y=at * A)
    _refused(_apply, _adapters(), y=6 * A + 2)
    _refused(_apply, _adapters(base_dtype=ft.FT_DT_F32), y=6 * A)  # base as another type
    _refused(_apply, _adapters(), work=_Buf(1 << 20, 7 * A))
    _refused(_apply, _adapters(), work=_Buf(1 << 20, 4 * A))
    _refused(_balanced, _balance(), w=3 * A)
    _refused(_balanced, _balance(), sel=A)
    _refused(_balanced, _balance(), loss=5 * A + 64)  # the last of the counts
    _refused(_balanced, _balance(), work=_Buf(1 << 20, A))
    _refused(_unbalanced, _balance(), dlogits=A + 64)
    for at in (2, 3, 4, 5, 6, 7):
        _refused(_unbalanced, _balance(), dlogits=at * A)


def test_nothing_to_do():
    assert _forward(_norm(), sum=None, y=None, codes=None, scale=None) == ft.FT_OK
    assert ft.ft_moe_rms_norm_forward(_norm(rows=0), None, None, None) == ft.FT_OK
    assert _backward(_norm(), dx=None, dresidual=None, dweight=None) == ft.FT_OK
    assert ft.ft_moe_rms_norm_backward(_norm(rows=0), None, None, None) == ft.FT_OK
    assert ft.ft_moe_adapters_apply(_adapters(tokens=0), None, None, None, None, None, None, None) == ft.FT_OK
    assert ft.ft_moe_balance_backward(_balance(tokens=0), None, None, None, None, None, None, None, None) == ft.FT_OK


def test_scratch_sizes_of_the_largest_calls():
    big = (1 << 24) - 1
    assert ft.ft_moe_rms_norm_work(_norm(rows=big, cols=big)) > 0
    assert ft.ft_moe_adapters_work(_adapters(tokens=big, rank=256)) >= big * 4
    assert ft.ft_moe_balance_work(_balance(tokens=big, experts=512)) > 0


def test_struct_layouts():
    from tests.test_abi import _c_layout

    structs = {t.__name__: t for t in (ft.ft_moe_rms_norm, ft.ft_moe_adapters, ft.ft_moe_balance)}
    c = _c_layout({n: [f for f, _ in t._fields_] for n, t in structs.items()})
    for n, t in structs.items():
        assert c[(n, "size")] == ctypes.sizeof(t), n
        for f, _ in t._fields_:
            assert c[(n, f)] == getattr(t, f).offset, (n, f)


def test_norms_ask_for_the_scratch_memory_they_use():
    """None for one or two rows that a workgroup holds, nor for any such rows without the weight's gradient."""
    for cols in (8, 7168, 16384):
        assert ft.ft_moe_rms_norm_work(_norm(rows=1, cols=cols)) == ft.ft_moe_rms_norm_work(_norm(rows=2, cols=cols)) == 0
        # a part for each row and column, no more
        assert ft.ft_moe_rms_norm_work(_norm(rows=4, cols=cols)) <= 4 * 4 * cols + 256
    for cols in (7, 16385):
        n = ft.ft_moe_rms_norm_work(_norm(rows=2, cols=cols))
        assert n > 0
        _refused(_backward, _norm(rows=2, cols=cols), work=_Buf(n - 1))
        _refused(_backward, _norm(rows=2, cols=cols), dweight=None, work=None)


def test_scratch_sizes_of_calls_without_tokens():
    """Asked for in a process of its own: a division by zero would end this one."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import lru_expert_cache_amd as ft\n"
            "for n in (1, 3, 4096):\n"
            "    for rank in (1, 16, 256):\n"
            "        assert ft.ft_moe_adapters_work(ft.make_adapters(ft.FT_DT_BF16, 0, 5000, 64, rank, n)) == 0\n"
            "        assert ft.ft_moe_adapters_work(ft.make_adapters(ft.FT_DT_F16, 0, 64, 64, rank, n, out_dtype=ft.FT_DT_F32)) == 0\n"
            "assert ft.ft_moe_rms_norm_work(ft.make_rms_norm(ft.FT_DT_BF16, 0, 32, 1e-6)) == 0\n"
            "assert ft.ft_moe_balance_work(ft.make_balance(ft.FT_DT_F32, 0, 16, 2, 0.01)) > 0\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120, cwd=root)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


def test_adapters_ask_for_the_scratch_memory_they_use():
    """One launch for both products keeps nothing in memory; two keep the sums of the first, at least."""
    for tokens in (1, 64):
        assert 0 < ft.ft_moe_adapters_work(_adapters(tokens=tokens, in_features=2048, rank=16)) <= 256
        assert ft.ft_moe_adapters_work(_adapters(tokens=tokens, in_features=2048, rank=17)) >= tokens * 17 * 4
    assert ft.ft_moe_adapters_work(_adapters(tokens=0)) == 0
