"""What the dense operators' host code decides, without a GPU: which kernels take which operands."""

import os
import subprocess

import pytest

import lru_expert_cache_amd as ft
from lru_expert_cache_amd import build

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
