"""How the few-rows attention cuts an item: each of its kernels works that out
for itself, so it must be a function of the lists alone, whatever a compiler
makes of the floating-point estimate in it.  The function is taken from the
kernel source and compiled for the host.  No GPU is needed."""
import ctypes as C
import os
import subprocess

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HOST = r"""
#include <algorithm>
#include <cmath>
using std::max;
using std::min;
#define __device__
#define __forceinline__ inline
// the quotient that the device's approximate division may return: its documented error is 2 ulp
static float skew;
static float __fdividef(float a, float b) { return (float)((double)a / (double)b * (1.0 + skew)); }
%s
extern "C" void parts(const int* tiles, const int* quota, int n, float by, int* out) {
    skew = by;
    for (int i = 0; i < n; ++i) out[i] = item_parts(tiles[i], quota[i]);
}
"""


def host_function(tmp_path):
    src = open(os.path.join(ROOT, "kv_cache_analyzer_b200", "csrc", "paged_decode.cu")).read()
    body = src[src.index("__device__ __forceinline__ int item_parts("):]
    body = body[:body.index("\n}\n") + 3]
    (tmp_path / "parts.cc").write_text(HOST % body)
    so = tmp_path / "parts.so"
    subprocess.check_call(["g++", "-O2", "-ffp-contract=off", "-shared", "-fPIC", "-o", so, tmp_path / "parts.cc"])
    f = C.CDLL(str(so)).parts
    f.argtypes = [C.c_void_p, C.c_void_p, C.c_int, C.c_float, C.c_void_p]
    return f


def test_an_items_parts_do_not_depend_on_the_approximate_quotient(tmp_path):
    f = host_function(tmp_path)
    gen = np.random.default_rng(0)
    # every small pair; multiples of the quota and their neighbours, quotas around a thousand above all; any pairs
    # (an item has at most 2^26 / 128 tiles)
    most = 2 ** 19
    pairs = [np.stack(np.meshgrid(np.arange(0, 400), np.arange(2, 80)), -1).reshape(-1, 2)]
    quota = np.concatenate([np.arange(2, 3000), gen.integers(2, most, 20000)])
    times = np.maximum(most // quota, 1)
    for k in (np.ones_like(quota), np.minimum(times, 74), np.minimum(times, 147), times):
        for by in (-2, -1, 0, 1, 2):
            pairs.append(np.stack([np.clip(k * quota + by, 0, most), quota], -1))
    pairs.append(np.stack([gen.integers(0, most + 1, 200000), gen.integers(2, most, 200000)], -1))
    pairs.append(np.stack([gen.integers(0, most + 1, 200000), gen.integers(2, 4000, 200000)], -1))
    pairs = np.concatenate(pairs)
    tiles, quota = (np.ascontiguousarray(pairs[:, i], dtype=np.int32) for i in (0, 1))
    want = -(-pairs[:, 0] // pairs[:, 1])
    for skew in (0.0, 2.0 ** -22, -2.0 ** -22):
        got = np.empty_like(tiles)
        f(tiles.ctypes.data, quota.ctypes.data, len(tiles), skew, got.ctypes.data)
        wrong = np.nonzero(got != want)[0]
        assert len(wrong) == 0, (skew, len(wrong), [(tiles[i], quota[i], got[i], want[i]) for i in wrong[:3]])
