"""The header in C and C++: the combine and its gradients count their rows' types differently, and the other call's
names do not compile."""
import os
import shutil
import subprocess

import pytest

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
CXX, CC = shutil.which("g++"), shutil.which("gcc")


def _compiles(body, compiler, lang):
    src = f'#include <mxmoe.h>\nint main(void) {{ {body} return 0; }}\n'
    r = subprocess.run([compiler, "-x", lang, "-Wall", "-Werror", "-fsyntax-only", "-I" + INCLUDE, "-"], input=src,
                       capture_output=True, text=True)
    return r.returncode == 0


def _combine(t):
    return f"moe_combine(0, {t}, 0, 0, 1, 1, 8, 0, 0, 0);"


def _backward(y, dy):
    return f"moe_combine_backward(0, 0, {y}, 0, 0, 1, 1, 8, 0, {dy}, 0, 0);"


TAKEN = [_combine("MOE_OUT_BF16"), _combine("MOE_OUT_FP16"), _combine("0"), "int32_t t = 1; " + _combine("t"),
         _backward("MOE_FLOAT_BF16", "MOE_FLOAT_FP32"), _backward("0", "1"), _backward("MOE_FLOAT_FP16", "0"),
         "int32_t t = 1; " + _backward("t", "t")]
MIXED = [_combine("MOE_FLOAT_BF16"), _combine("MOE_FLOAT_FP32"), _backward("MOE_OUT_BF16", "MOE_FLOAT_BF16"),
         _backward("MOE_FLOAT_BF16", "MOE_OUT_BF16"), _backward("MOE_OUT_BF16", "MOE_OUT_BF16"),
         _backward("MOE_OUT_FP32", "0"), _backward("0", "MOE_OUT_FP32")]


@pytest.mark.skipif(CXX is None, reason="no C++ compiler")
@pytest.mark.parametrize("body", TAKEN)
def test_each_calls_own_types_compile(body):
    assert _compiles(body, CXX, "c++")
    assert CC is None or _compiles(body, CC, "c")


@pytest.mark.skipif(CXX is None, reason="no C++ compiler")
@pytest.mark.parametrize("body", MIXED)
def test_the_other_calls_types_do_not_compile(body):
    assert not _compiles(body, CXX, "c++")
