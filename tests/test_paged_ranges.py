"""The rows, keys and groups that the paged operators give a sequence
(csrc/paged_ranges.h), compiled for the host and compared with unbounded integers:
no value that the caller's int32 arrays can hold names a row or a key outside."""
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
#include "paged_ranges.h"
extern "C" void ranges(const int32_t* cu_q, const int32_t* kv_len, const int32_t* prefix, int n, int q_rows, int capacity,
                       int max_prefix, int max_kv, int shift, int32_t* out) {
  for (int b = 0; b < n; ++b) {
    const moe::PagedRange s = moe::paged_range(cu_q, kv_len, b, q_rows, capacity, prefix[b], max_prefix, max_kv, shift);
    out[6 * b] = s.q0, out[6 * b + 1] = s.lq, out[6 * b + 2] = s.own, out[6 * b + 3] = s.end;
    out[6 * b + 4] = s.lq ? moe::last_key(s, 0) : -1, out[6 * b + 5] = s.lq ? moe::last_key(s, s.lq - 1) : -1;
  }
}
extern "C" void groups(const int32_t* cu, int n, int n_seqs, int32_t* out) {
  for (int g = 0; g < n; ++g) {
    const moe::GroupRange r = moe::group_range(cu, g, n_seqs);
    out[2 * g] = r.first, out[2 * g + 1] = r.past;
  }
}
"""
EDGES = [LOW, LOW + 1, -5, -1, 0, 1, 5, 8, 9, 63, 64, 100, HIGH - 1, HIGH]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("ranges")
    src, so = str(d / "ranges.cpp"), str(d / "ranges.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    # a signed overflow ends the process
    subprocess.run([gxx, "-O1", "-ftrapv", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", so], check=True)
    return ctypes.CDLL(so)


def _p(a):
    return a.ctypes.data_as(ctypes.c_void_p)


@pytest.mark.parametrize("q_rows,capacity,max_prefix,max_kv,shift", [
    (8, 64, 64, 64, 4), (8, 64, 30, 20, 4), (262144, (1 << 30) - 64, (1 << 30) - 64, (1 << 30) - 64, 6), (40, 0, 0, 0, 5),
    (40, 128, 0, 128, 7), (40, 1024, 1000, 3, 6)])
def test_every_value_stays_inside(lib, q_rows, capacity, max_prefix, max_kv, shift):
    cu = np.asarray([v for pair in itertools.product(EDGES, EDGES) for v in pair], np.int32)
    n = len(cu) - 1
    g = np.random.default_rng(7)
    length, prefix = g.choice(np.asarray(EDGES, np.int32), n), g.choice(np.asarray(EDGES, np.int32), n)
    out = np.empty((n, 6), np.int32)
    lib.ranges(_p(cu), _p(length), _p(prefix), n, q_rows, capacity, max_prefix, max_kv, shift, _p(out))
    q0, lq, own, end, first, last = out.astype(np.int64).T
    a, b = np.clip(cu[:-1].astype(np.int64), 0, q_rows), np.clip(cu[1:].astype(np.int64), 0, q_rows)
    assert np.array_equal(q0, a) and np.array_equal(lq, np.maximum(b - a, 0))
    pre = np.minimum(np.maximum(prefix.astype(np.int64), 0), max_prefix)
    lk = np.maximum(length.astype(np.int64), 0)
    assert np.array_equal(own, pre >> shift << shift) and np.all(own <= capacity)
    assert np.array_equal(end, np.minimum(np.minimum(lk, capacity), pre + max_kv))
    some = lq > 0
    assert np.array_equal(first[some], np.minimum(lk - lq, end - 1)[some])
    assert np.array_equal(last[some], np.minimum(lk - 1, end - 1)[some])


def test_groups_stay_inside(lib):
    cu = np.asarray([v for pair in itertools.product(EDGES, EDGES) for v in pair], np.int32)
    for n_seqs in (0, 1, 7, 65536):
        out = np.empty((len(cu) - 1, 2), np.int32)
        lib.groups(_p(cu), len(cu) - 1, n_seqs, _p(out))
        first = np.clip(cu[:-1].astype(np.int64), 0, n_seqs)
        assert np.array_equal(out[:, 0], first)
        assert np.array_equal(out[:, 1], np.maximum(np.clip(cu[1:].astype(np.int64), 0, n_seqs), first))


WORK = """
#define __host__
#define __device__
#include "paged_ranges.h"
extern "C" int work(int split, int splits, int slots, int every_slot) {
  return static_cast<int>(moe::split_work(split, splits, slots, every_slot));
}
"""
ATTEND, EMPTY, NOTHING = range(3)


def test_shares_of_a_row(tmp_path):
    """A row of one share never has one in the workspace, and its output is written by exactly one block; of several, where
    the join reads them all, every one is written."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("needs g++")
    src, so = str(tmp_path / "work.cpp"), str(tmp_path / "work.so")
    with open(src, "w") as f:
        f.write(WORK)
    subprocess.run([gxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", so], check=True)
    work = ctypes.CDLL(so).work
    for slots in range(1, 6):
        for launched in range(1, slots + 1):  # splits of the launch; the other slots are a prefix's
            for splits in range(launched + 1):  # that the tile has keys for
                done = [work(s, splits, slots, 1) for s in range(launched)]
                if slots == 1:
                    assert done == [ATTEND]
                else:
                    assert done == [ATTEND] * splits + [EMPTY] * (launched - splits)
                some = max(splits, 1)  # without groups the join reads the splits that there are
                assert [work(s, splits, slots, 0) for s in range(launched)] == [ATTEND] * some + [NOTHING] * (launched - some)
