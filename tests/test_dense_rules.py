"""What the dense operators' host code decides, without a GPU: which kernels take which operands."""

import os
import subprocess

import pytest

import lru_expert_cache_amd as ft
from lru_expert_cache_amd import build
from tests import dense_exact as de

# DenseForm
GATED, ROWS, GRAD, COLS, OUTER, INT, INT_GATED = range(7)


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    ft.lib()
    exe = str(tmp_path_factory.mktemp("dense") / "dense_check")
    cmd = [build.HIPCC] + build.COMMON + ["-I", build.CSRC, os.path.join(build.ROOT, "tests", "native", "dense_check.cpp"),
                                          "-L", build.PKG, "-l:libftmoe.so", f"-Wl,-rpath,{build.PKG}", "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(*args):
        r = subprocess.run([exe] + [str(a) for a in args], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        return r.stdout.split()

    return run


@pytest.mark.parametrize("form", [INT, INT_GATED])
@pytest.mark.parametrize("tokens", [ft.FT_DT_BF16, ft.FT_DT_F16, ft.FT_DT_F32, 4, -1])
def test_only_the_token_types_of_a_form_are_quantised(check, form, tokens):
    """The down product has fp32 rows to quantise, the gated product 16-bit ones: another type is refused, not read as
    that one."""
    fits = {INT: [ft.FT_DT_F32], INT_GATED: [ft.FT_DT_BF16, ft.FT_DT_F16]}[form]
    assert check("few", form, tokens) == ["taken" if tokens in fits else "refused"]


@pytest.mark.parametrize("form", [GATED, ROWS])
def test_16_bit_products_quantise_nothing(check, form):
    assert check("few", form, ft.FT_DT_F32) == ["refused"]


def test_tiles_of_the_sizes_that_are_compared_bit_for_bit(check):
    """The plan sends these sizes to 256 x 256 tiles, with K whole and in parts, dx and the weight gradients together and
    apart: if it changes, sizes that cover those kernels take their place."""
    def plans(T, H, I):
        p = {"gated": check("plan", GATED, T, I, H, 1), "rows": check("plan", ROWS, T, H, I, 1), "dh": check("plan", GRAD, T, I, H, 1),
             "dx": check("plan", COLS, T, H, I, 2), "dw": check("plan", OUTER, I, H, T, 1, I, H, T, 1, H, I, T, 1),
             "int": check("plan", INT, T, H, I, 1), "int gated": check("plan", INT_GATED, T, I, H, 1)}
        pair = check("pair", I, H, T, I, H, T, H, I, T, T, H, I)
        return {n: (int(v[0]), int(v[1])) for n, v in p.items()}, int(pair[0])

    for size in de.TILED[:2]:
        p, pair = plans(*size)
        assert set(p.values()) == {(256, 1)} and pair == 256, (size, p, pair)
    p, pair = plans(*de.TILED[2])
    assert p["gated"] == p["rows"] == p["dx"] == p["dw"] == (256, 1) and p["dh"][0] == 256 and p["dh"][1] > 1 and pair == 256
    p, _ = plans(*de.TILED[3])
    assert p["dx"][0] == 256 and p["dx"][1] > 1
    p, _ = plans(*de.TILED[4])
    assert p["dw"][0] == 256 and p["dw"][1] > 1
    p, pair = plans(*de.TILED[5])
    assert p["dx"] == p["dw"] == (256, 1) and pair == 0
    for T, K, N in de.PRODUCTS[3:5]:
        assert check("plan", INT, T, N, K, 1) == ["256", "1"]
    assert {check("plan", INT, T, N, K, 1)[0] for T, K, N in de.PRODUCTS if T > 64} == {"128", "256"}
