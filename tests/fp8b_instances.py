"""Which kernel a size of the block-scaled fp8 products takes, from the library's own rule
(csrc/qpl_fp8b_shape.h compiled for the host), so that the tests can say that they reach every kernel."""
import ctypes
import functools
import os
import subprocess
import tempfile

from conftest import ROOT

SHIM = """
#include "qpl_fp8b_shape.h"
using namespace qpl;
extern "C" int shapes() { return kFp8bShapeCount; }
extern "C" int ungated(int v) { return !fp8b_gated_shape(v); }
extern "C" int shape(int64_t M, int64_t K, int64_t N, int segs, int gated) {
  return segs == 1 && fp8b_token_fits(M, K) ? -1 : fp8b_shape(M, (K + 127) / 128 * segs, N, gated != 0);
}
"""


@functools.lru_cache(maxsize=None)
def rule():
    csrc = os.path.join(ROOT, "precision_quantized_linear_amd", "csrc")
    with tempfile.TemporaryDirectory() as d:
        so = os.path.join(d, "rule.so")
        subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", csrc, "-x", "c++", "-", "-o", so],
                       input=SHIM, text=True, check=True)
        lib = ctypes.CDLL(so)
    lib.shape.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2
    return lib


def linear(M, K, N):
    """-1: few rows in one launch, else the number of the shape."""
    return rule().shape(M, K, N, 1, 0)


def gated(M, K, H):
    return rule().shape(M, K, 2 * H, 1, 1)


def pair(M, H, K):
    """The product of the gated backward: two segments of H."""
    return rule().shape(M, H, K, 2, 0)


def every(gated=False):
    return {v for v in range(rule().shapes()) if not (gated and rule().ungated(v))}
