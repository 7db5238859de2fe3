"""Dense feed-forward operators without a GPU: refusals that come before any
device call, scratch sizes, and calls that have nothing to do."""

import ctypes

import pytest

import lru_expert_cache_amd as ft

A = 1 << 20  # an address that is never read: every call here is refused before it would be


def _refused(call, *args, **kw):
    with pytest.raises(ft.FtError) as e:
        call(*args, **kw)
    assert e.value.code == ft.FT_E_INVALID
    assert ft.ft_moe_last_error()


class _Buf:
    def __init__(self, n, at=64 * A):
        self.n, self.at = n, at

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n

    def element_size(self):
        return 1


def _ffn(**kw):
    d = dict(dtype=ft.FT_DT_BF16, tokens=4, hidden=32, inter=16)
    d.update(kw)
    return ft.make_gated_ffn(**d)


BAD_FFN = [dict(dtype=ft.FT_DT_F32), dict(dtype=0), dict(tokens=-1), dict(hidden=0), dict(inter=0), dict(hidden=1 << 24),
           dict(tokens=1 << 24), dict(ld_x=31), dict(ld_y=8), dict(ld_gu=31), dict(ld_w_in=31), dict(ld_w_out=15),
           dict(ld_x=1 << 32), dict(ld_x=-5)]


@pytest.mark.parametrize("kw", BAD_FFN)
def test_bad_block_descriptions(kw):
    d = _ffn(**kw)
    _refused(ft.ft_moe_gated_ffn_work, d)
    _refused(ft.ft_moe_gated_ffn_forward, d, A, 2 * A, 3 * A, 4 * A, 5 * A, None, _Buf(1 << 20))
    _refused(ft.ft_moe_gated_ffn_backward, d, A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A, None, None, None, _Buf(1 << 20))
    _refused(ft.ft_moe_int_gated_ffn, d, A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A, 8 * A, _Buf(1 << 20))


def test_scratch_memory_is_checked():
    d = _ffn()
    n = ft.ft_moe_gated_ffn_work(d)
    assert n > 0 and ft.ft_moe_gated_ffn_work(d, True) > n
    args = (d, A, 2 * A, 3 * A, 4 * A, 5 * A, None)
    _refused(ft.ft_moe_gated_ffn_forward, *args, _Buf(n - 1))
    _refused(ft.ft_moe_gated_ffn_forward, *args, None)
    _refused(ft.ft_moe_gated_ffn_forward, *args, _Buf(n, 64 * A + 8))  # not 16-byte aligned
    nb = ft.ft_moe_gated_ffn_work(d, True)
    _refused(ft.ft_moe_gated_ffn_backward, d, A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A, 8 * A, 9 * A, 10 * A, _Buf(nb - 1))
    ni = ft.ft_moe_int_gated_ffn_work(d)
    _refused(ft.ft_moe_int_gated_ffn, d, A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A, 8 * A, _Buf(ni - 1))
    L = ft.lib()
    assert L.ft_moe_gated_ffn_work(ctypes.byref(d), 0, None) == ft.FT_E_INVALID
    assert L.ft_moe_int_gated_ffn_work(ctypes.byref(d), None) == ft.FT_E_INVALID
    assert L.ft_moe_int_matmul_work(None, None) == ft.FT_E_INVALID


@pytest.mark.parametrize("at", range(5))
def test_block_pointers_are_checked(at):
    d = _ffn()
    for value in (None, A + 1):  # missing; not aligned to an element
        p = [(i + 2) * A for i in range(5)]
        p[at] = value
        _refused(ft.ft_moe_gated_ffn_forward, d, *p, None, _Buf(1 << 20))


def test_arguments_given_twice():
    d, w = _ffn(), _Buf(1 << 20)
    _refused(ft.ft_moe_gated_ffn_forward, d, A, 2 * A, 3 * A, 4 * A, A, None, w)  # y is x
    _refused(ft.ft_moe_gated_ffn_forward, d, A, 2 * A, 3 * A, 4 * A, 5 * A, 5 * A, w)  # gu is y
    _refused(ft.ft_moe_gated_ffn_forward, d, A, 2 * A, 3 * A, 4 * A, 5 * A, w.at, w)  # gu is the scratch memory
    p = [d, A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A]
    _refused(ft.ft_moe_gated_ffn_backward, *p, A, None, None, None, w)  # dx is x
    _refused(ft.ft_moe_gated_ffn_backward, *p, 7 * A, 8 * A, 8 * A, 9 * A, w)  # two gradients in one place
    _refused(ft.ft_moe_gated_ffn_backward, *p, 7 * A, 8 * A, None, 9 * A, w)  # gradients given in part
    _refused(ft.ft_moe_int_quantize, ft.FT_DT_BF16, 2, 16, A, A, 2 * A)
    m = ft.make_int_matmul(2, 16, 16, ft.FT_DT_BF16)
    _refused(ft.ft_moe_int_matmul, m, A, 2 * A, 3 * A, 4 * A, A, w)


@pytest.mark.parametrize("kw", [dict(out_dtype=0), dict(out_dtype=4), dict(tokens=-1), dict(in_features=0),
                                dict(in_features=131072), dict(out_features=0), dict(ld_x=15), dict(ld_w=15), dict(ld_y=7)])
def test_bad_products(kw):
    d = dict(tokens=2, in_features=16, out_features=8, out_dtype=ft.FT_DT_BF16)
    d.update(kw)
    d = ft.make_int_matmul(**d)
    _refused(ft.ft_moe_int_matmul_work, d)
    _refused(ft.ft_moe_int_matmul, d, A, 2 * A, 3 * A, 4 * A, 5 * A, _Buf(1 << 20))


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(dtype=9), dict(rows=-1), dict(cols=0), dict(ld_x=15), dict(ld_codes=3)])
def test_bad_quantisation(kw):
    d = dict(dtype=ft.FT_DT_BF16, rows=2, cols=16, x=A, codes=2 * A, scale=3 * A)
    d.update(kw)
    _refused(ft.ft_moe_int_quantize, **d)


def test_long_rows_do_not_fit_32_bit_sums():
    _refused(ft.ft_moe_int_gated_ffn_work, _ffn(hidden=131072))
    _refused(ft.ft_moe_int_gated_ffn_work, _ffn(inter=131072))
    assert 127 * 127 * 131071 < 2**31


def test_no_tokens_is_no_work():
    d = _ffn(tokens=0)
    assert ft.ft_moe_gated_ffn_forward(d, None, None, None, None, None) == ft.FT_OK
    assert ft.ft_moe_gated_ffn_backward(d, None, None, None, None, None, None) == ft.FT_OK
    assert ft.ft_moe_int_gated_ffn(d, None, None, None, None, None, None, None, None) == ft.FT_OK
    assert ft.ft_moe_int_quantize(ft.FT_DT_F16, 0, 16, None, None, None) == ft.FT_OK
    assert ft.ft_moe_int_matmul(ft.make_int_matmul(0, 16, 8, ft.FT_DT_F32), None, None, None, None, None) == ft.FT_OK


def test_struct_layouts():
    from tests.test_abi import _c_layout

    structs = {"ft_moe_gated_ffn": ft.ft_moe_gated_ffn, "ft_moe_int_product": ft.ft_moe_int_product}
    c = _c_layout({n: [f for f, _ in t._fields_] for n, t in structs.items()})
    for n, t in structs.items():
        assert c[(n, "size")] == ctypes.sizeof(t), n
        for f, _ in t._fields_:
            assert c[(n, f)] == getattr(t, f).offset, (n, f)


@pytest.mark.parametrize("hidden,inter", [(17, 19), (2721, 1043), (16, 19), (17, 16), (1, 1)])
@pytest.mark.parametrize("backward", [False, True])
def test_scratch_memory_holds_copies_of_rows_that_are_no_whole_pieces(hidden, inter, backward):
    """Rows that are not multiples of 16 bytes are copied to rows that are: the scratch memory has room for them."""
    for tokens in (1, 33, 500):
        odd = ft.ft_moe_gated_ffn_work(_ffn(tokens=tokens, hidden=hidden, inter=inter), backward)
        up = lambda v: -(-v // 64) * 64
        h, i = up(hidden), up(inter)
        own = tokens * i * 2 * (3 if backward else 1)
        copies = (tokens * h * (2 if backward else 1) + 2 * inter * h) * 2 if hidden % 8 else 0
        copies += hidden * i * 2 if inter % 8 else 0
        assert odd >= own + copies
        assert ft.ft_moe_int_gated_ffn_work(_ffn(tokens=tokens, hidden=hidden, inter=inter)) >= tokens * (hidden + 5 * inter)
    assert ft.ft_moe_gated_ffn_work(_ffn(tokens=0, hidden=hidden, inter=inter), backward) >= 0


def test_scratch_memory_that_is_an_input():
    d, w = _ffn(), _Buf(1 << 20)
    for at in range(4):
        p = [A, 2 * A, 3 * A, 4 * A]
        p[at] = w.at
        _refused(ft.ft_moe_gated_ffn_forward, d, *p, 5 * A, None, w)
    m = ft.make_int_matmul(2, 17, 16, ft.FT_DT_BF16)  # rows that are copied
    assert ft.ft_moe_int_matmul_work(m) > 0
    _refused(ft.ft_moe_int_matmul, m, w.at, 2 * A, 3 * A, 4 * A, 5 * A, w)
    _refused(ft.ft_moe_int_matmul, m, A, 2 * A, w.at, 4 * A, 5 * A, w)
