"""Which kernel a size of the 8-bit integer products takes, from the library's own rule
(csrc/qpl_int8_shape.h compiled for the host), so that the tests can say that they reach every kernel."""
import ctypes
import functools
import os
import subprocess
import tempfile

from conftest import ROOT

TOKEN = "token"
NAMES = ("16x16", "16x32", "32x32", "64x64", "64x128", "128x128 four stages", "128x256", "256x256",
         "128x128 two stages")

SHIM = """
#include "qpl_int8_shape.h"
using namespace qpl;
static int64_t tiles(int v, int64_t M) { return (M + kShapes[v].rows - 1) / kShapes[v].rows; }
static int instance(int v, int64_t row_tiles, int64_t N) { return v == 5 && !four_stages(row_tiles, N) ? 8 : v; }
extern "C" int dense(int64_t M, int64_t K, int64_t N) {
  if (token_fits(M, K)) return -1;
  const int v = dense_shape(M, K, N);
  return instance(v, tiles(v, M), N);
}
extern "C" int grouped(int64_t R, int64_t K, int64_t N, int64_t E) {
  const int v = grouped_shape(R, K, N, E);
  return instance(v, row_tile_bound(R, E, kShapes[v].rows), N);
}
extern "C" int split(int64_t rows, int64_t K, int gathered) { return split_rows(rows, K, gathered != 0); }
"""


@functools.lru_cache(maxsize=None)
def rule():
    csrc = os.path.join(ROOT, "precision_quantized_linear_amd", "csrc")
    with tempfile.TemporaryDirectory() as d:
        so = os.path.join(d, "rule.so")
        subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", csrc, "-x", "c++", "-", "-o", so],
                       input=SHIM, text=True, check=True)
        lib = ctypes.CDLL(so)
    lib.dense.argtypes = [ctypes.c_int64] * 3
    lib.grouped.argtypes = [ctypes.c_int64] * 4
    lib.split.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    return lib


def dense(M, K, N):
    v = rule().dense(M, K, N)
    return TOKEN if v < 0 else NAMES[v]


def grouped(R, K, N, E):
    return NAMES[rule().grouped(R, K, N, E)]


def split(rows, K, gathered):
    """Does the row quantizer take a workgroup per row (or a wavefront)?"""
    return bool(rule().split(rows, K, gathered))
