"""The search for a bound that k keys reach (csrc/bound_search.h), compiled for
the host: it ends, in few rounds, whatever range it is given."""

from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest

from conftest import ROOT

SOURCE = r"""
#include <cstddef>
#include "bound_search.h"
using namespace gemm_f32_impl;
// The bound; *rounds: counts made (-1: a bin outside the histogram).
extern "C" uint32_t search(const uint32_t* keys, int n, int k, uint32_t low,
                           uint32_t high, int enough, int* rounds) {
  *rounds = 0;
  auto count = [&](uint32_t low, uint32_t high, int shift, int& in_step) {
    int hist[kBoundBins] = {0};
    for (int i = 0; i < n; ++i) {
      if (keys[i] < low) continue;
      const uint32_t bin = bound_bin(keys[i], low, high, shift);
      if (bin >= kBoundBins || *rounds < 0) { *rounds = -1; return 0; }
      ++hist[bin];
    }
    ++*rounds;
    int b = kBoundBins - 1, before = 0;
    while (b > 0 && before + hist[b] < k) before += hist[b--];
    in_step = hist[b];
    return b;
  };
  return bound_search(low, high, enough, count);
}
"""

LOWEST = 0x007fffff  # -Inf in the order of the floats


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    where = tmp_path_factory.mktemp("search")
    src, out = where / "search.cpp", where / "search.so"
    src.write_text(SOURCE)
    subprocess.run(
        ["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared",
         "-I", os.path.join(ROOT, "dense_fp32_matrix_02_gb300", "csrc"),
         str(src), "-o", str(out)], check=True)
    fn = ctypes.CDLL(str(out)).search
    u32 = ctypes.c_uint32
    fn.restype = u32
    fn.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, u32, u32,
                   ctypes.c_int, ctypes.POINTER(ctypes.c_int)]

    def run(keys, k, low, high, enough=32):
        keys = np.ascontiguousarray(keys, dtype=np.uint32)
        rounds = ctypes.c_int()
        got = fn(keys.ctypes.data, keys.size, k, int(low), int(high), enough,
                 ctypes.byref(rounds))
        assert 1 <= rounds.value <= 4
        return got

    return run


def order(f):
    u = np.asarray(f, np.float32).view(np.uint32)
    return np.where(u >> 31, ~u, u | np.uint32(0x80000000)).astype(np.uint32)


@pytest.mark.parametrize("n,k", [(1, 1), (28, 28), (700, 28), (3000, 28),
                                 (20000, 264)])
def test_bound_of_keys_in_the_range(search, n, k):
    """k keys reach the bound, and of random ones few more."""
    rng = np.random.default_rng(n)
    for scale in (2.0, 1e-30, 1e30):
        keys = order(rng.standard_normal(n) * scale)
        for low in (LOWEST, keys.min()):
            got = search(keys, k, low, keys.max())
            assert k <= (keys >= got).sum() <= k + 31


@pytest.mark.parametrize("n,k", [(700, 28), (3000, 28), (20000, 264)])
@pytest.mark.parametrize("high", [-3e38, -1.0, 0.0, 1e-38, 0.5, 3.0, 3e38])
def test_range_that_ends_below_the_keys(search, n, k, high):
    """Maxima that belong to other logits: the search ends, and k keys reach
    the bound."""
    rng = np.random.default_rng(k)
    for _ in range(20):
        keys = order(rng.standard_normal(n) * 2)
        got = search(keys, k, LOWEST, order(high))
        assert got <= max(int(order(high)), LOWEST)
        assert (keys >= got).sum() >= k


def test_any_keys_and_ranges(search):
    rng = np.random.default_rng(7)
    for _ in range(300):
        n = int(rng.integers(1, 400))
        keys = rng.integers(0, 2**32, n, dtype=np.uint64)
        keys >>= np.uint64(rng.integers(0, 33))
        low, high = (int(v) for v in rng.integers(0, 2**32, 2))
        search(keys, int(rng.integers(1, n + 1)), low, high,
               int(rng.integers(0, 40)))


def test_equal_keys_and_ends(search):
    for v in (0, LOWEST, 0x80000000, 2**32 - 1):
        keys = np.full(500, v, np.uint32)
        assert search(keys, 20, v, v) == v
        assert search(keys, 20, 0, 2**32 - 1) == v
    keys = np.arange(2**32 - 1000, 2**32, dtype=np.uint64)
    got = search(keys, 5, 0, 2**32 - 1, 0)
    assert got == 2**32 - 5
