"""qpl_timing_collect and programs built against a header with fewer kernel kinds: the
exported function writes the kinds it began with, the counted one what its caller has room for."""
import ctypes
import os
import re
import subprocess

import pytest

import precision_quantized_linear_amd as qpl
from conftest import ROOT

OK, NULL, ARG = 0, 1, 4
FIRST = 18


@pytest.fixture(scope="module")
def lib():
    return qpl.load()


def arrays(n):
    return (ctypes.c_int64 * n)(*[7] * n), (ctypes.c_double * n)(*[7.0] * n)


def test_the_uncounted_call_stays_inside_the_first_kinds(lib):
    a, b = arrays(64)
    assert lib.qpl_timing_collect(ctypes.cast(a, ctypes.c_void_p), ctypes.cast(b, ctypes.c_void_p)) == OK
    assert list(a) == [0] * FIRST + [7] * (64 - FIRST) and list(b) == [0.0] * FIRST + [7.0] * (64 - FIRST)


@pytest.mark.parametrize("count", [0, 1, FIRST, len(qpl.KERNELS), 40])
def test_the_counted_call_writes_that_many(lib, count):
    a, b = arrays(64)
    assert lib.qpl_timing_collect_n(ctypes.cast(a, ctypes.c_void_p), ctypes.cast(b, ctypes.c_void_p), count) == OK
    assert list(a) == [0] * count + [7] * (64 - count) and list(b) == [0.0] * count + [7.0] * (64 - count)


def test_counted_refusals(lib):
    a, b = arrays(4)
    assert lib.qpl_timing_collect_n(None, ctypes.cast(b, ctypes.c_void_p), 4) == NULL
    assert lib.qpl_timing_collect_n(ctypes.cast(a, ctypes.c_void_p), None, 4) == NULL
    assert lib.qpl_timing_collect_n(ctypes.cast(a, ctypes.c_void_p), ctypes.cast(b, ctypes.c_void_p), -1) == ARG


def test_source_passes_its_own_count():
    header = open(os.path.join(ROOT, "include", "qpl.h")).read()
    assert int(re.search(r"QPL_KERNEL_COUNT = (\d+)", header).group(1)) == len(qpl.KERNELS)
    code = ("#include <qpl.h>\nint f(void) { int64_t n[QPL_KERNEL_COUNT]; double t[QPL_KERNEL_COUNT];\n"
            "return qpl_timing_collect(n, t); }\n")
    for lang in ("c", "c++"):
        r = subprocess.run(["g++", "-x", lang, "-E", "-P", "-I", os.path.join(ROOT, "include"), "-"], input=code,
                           capture_output=True, text=True, check=True)
        assert "qpl_timing_collect_n((n), (t), QPL_KERNEL_COUNT)" in r.stdout
        subprocess.run(["g++", "-x", lang, "-fsyntax-only", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-"],
                       input=code, text=True, check=True)


@pytest.mark.gpu
def test_every_kind_is_collected():
    import torch
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    lib = qpl.load()
    qpl.timing_enable(True)
    try:
        qpl.quant_act_int8(x)
        qpl.quant_act_fp8_row(x)
        got = qpl.timing_collect()
        qpl.quant_act_int8(x)
        qpl.quant_act_fp8_row(x)
    finally:
        qpl.timing_enable(False)
    assert {k for k, (n, _) in got.items() if n} == {"quant_int8", "quant_fp8_row"}
    a, b = arrays(64)
    assert lib.qpl_timing_collect(ctypes.cast(a, ctypes.c_void_p), ctypes.cast(b, ctypes.c_void_p)) == OK
    assert list(a) == [1] + [0] * (FIRST - 1) + [7] * (64 - FIRST)
    assert all(v == (0, 0.0) for v in qpl.timing_collect().values())    # the other kinds' records are cleared too
