"""The rows and keys that moe_attention gives a sequence (csrc/attention_ranges.h),
compiled for the host and compared with unbounded integers: no value that the
caller's int32 arrays can hold names a row outside the tensors."""
import ctypes
import itertools
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_routed_expert_moe_amd", "csrc")
LOW, HIGH = -(1 << 31), (1 << 31) - 1
SOURCE = """
#define __host__
#define __device__
#include "attention_ranges.h"
extern "C" void ranges(const int32_t* cu_q, const int32_t* kv_start, const int32_t* kv_len, int n, int q_rows, int kv_rows,
                       int max_kv, int32_t* out) {
  for (int b = 0; b < n; ++b) {
    const moe::SeqRange s = moe::seq_range(cu_q, kv_start, kv_len, b, q_rows, kv_rows, max_kv);
    out[4 * b] = s.q0, out[4 * b + 1] = s.lq, out[4 * b + 2] = s.k0, out[4 * b + 3] = s.lk;
  }
}
extern "C" int last(const int32_t* cu_q, const int32_t* kv_start, const int32_t* kv_len, int q_rows, int kv_rows,
                    int max_kv, int causal, int pos) {
  return moe::last_key(moe::seq_range(cu_q, kv_start, kv_len, 0, q_rows, kv_rows, max_kv), causal, pos);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("ranges")
    src, so = str(d / "ranges.cpp"), str(d / "ranges.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    # -fwrapv: an overflow wraps, as the GPU's integers do
    subprocess.run([gxx, "-O1", "-fwrapv", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", so], check=True)
    return ctypes.CDLL(so)


def _ranges(lib, cu, start, length, q_rows, kv_rows, max_kv):
    a = [None if v is None else np.asarray(v, np.int32) for v in (cu, start, length)]
    out = np.empty((len(cu) - 1, 4), np.int32)
    p = lambda v: None if v is None else v.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    lib.ranges(*map(p, a), len(cu) - 1, q_rows, kv_rows, max_kv, p(out))
    return out.astype(np.int64)


EDGES = [LOW, LOW + 1, LOW + 7, -5, -1, 0, 1, 5, 7, 8, 9, 100, HIGH - 1, HIGH]


@pytest.mark.parametrize("q_rows,kv_rows,max_kv", [(8, 8, 8), (8, 100, 60), (40, 3, 3), (8, 0, 0), (262144, HIGH, HIGH)])
def test_every_value_stays_inside_the_tensors(lib, q_rows, kv_rows, max_kv):
    cu = [v for pair in itertools.product(EDGES, EDGES) for v in pair]  # every ordered pair of values, one after the other
    n = len(cu) - 1
    g = np.random.default_rng(7)
    for start, length in ((None, None), (g.choice(EDGES, n), g.choice(EDGES, n))):
        q0, lq, k0, lk = _ranges(lib, cu, start, length, q_rows, kv_rows, max_kv).T
        a = np.clip(np.asarray(cu[:-1], np.int64), 0, q_rows)
        b = np.clip(np.asarray(cu[1:], np.int64), 0, q_rows)
        assert np.array_equal(q0, a) and np.array_equal(lq, np.maximum(b - a, 0))
        assert np.all(q0 >= 0) and np.all(q0 + lq <= q_rows)
        assert np.all(k0 >= 0) and np.all(lk >= 0) and np.all(k0 + lk <= kv_rows) and np.all(lk <= max_kv)


@pytest.mark.parametrize("cache", [False, True])
def test_last_key_hangs_on_the_lengths_as_given(lib, cache):
    """Key j is seen where j <= i + Lk - Lq (causal) and where it is there: inside Lk, k's rows and max_kv."""
    p = lambda v: np.asarray(v, np.int32).ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    for lq, lk, k0, kv_rows, max_kv in itertools.product((1, 5, 9), (0, 1, 5, 7, 12, HIGH), (0, 3), (0, 4, 20), (0, 3, 6, 20)):
        if not cache:
            lk, k0 = lq, 2
        for causal, i in itertools.product((0, 1), range(lq)):
            got = lib.last(p([2, 2 + lq]), p([k0]) if cache else None, p([lk]) if cache else None, 2 + lq, kv_rows, max_kv,
                           causal, i)
            there = min(lk, max(kv_rows - k0, 0), max_kv)
            seen = [j for j in range(there) if not causal or j <= i + lk - lq]
            assert max(got, -1) == max(seen, default=-1), (lq, lk, k0, kv_rows, max_kv, causal, i)
