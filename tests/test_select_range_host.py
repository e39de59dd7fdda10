"""The boundary search of the eviction, run on the host: the same steps, keys and float
compares that the kernel uses (csrc/select_range.cuh), against a sort.  Nothing here needs a
GPU.  What is checked: the search ends, its counts are exact, and exactly the wanted number
of scores lies at or above the boundary, for scores with NaN, infinities, zeros of both
signs, denormals and many ties, whatever range a sample proposes."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from sparse_selection_primitive_b200 import _build

SOURCE = r"""
#include <algorithm>
#include <vector>
#include "select_range.cuh"
using namespace lapsum;

struct Row {
    const float* x;
    int competitors, need;
    Range g;
    std::vector<int> list;
    std::vector<char> above;
    int marks = 0, narrows = 0;

    Range range() const { return g; }
    void set(Range r) { g = r; }
    Range mark() {
        const RangeTest is = range_test(g);
        Range r{g.lo, g.hi, 0, 0};
        list.clear();
        above.assign(competitors, 0);
        ++marks;
        for (int i = 0; i < competitors; ++i) {
            const bool over = x[i] >= is.over, in = (is.all || x[i] >= is.floor) && !over;
            above[i] = over;
            r.above += over;
            r.inside += in;
            if (in && (int)list.size() < kSelList) list.push_back(i);
        }
        return r;
    }
    template <class Get>
    void narrow_by(int n, Get get) {
        std::vector<int> hist(kSelBins, 0);
        const int shift = range_shift(g.lo, g.hi);
        for (int i = 0; i < n; ++i) {
            const uint32_t key = score_key(get(i));
            if (key >= g.lo && key <= g.hi) ++hist.at((key - g.lo) >> shift);
        }
        int at = g.above;
        for (int b = kSelBins - 1; b >= 0; --b) {
            if (at < need && need <= at + hist[b]) {
                g = range_of_bin(g, b, at, hist[b]);
                return;
            }
            at += hist[b];
        }
    }
    void narrow() {
        ++narrows;
        narrow_by(competitors, [&](int i) { return x[i]; });
    }
};

extern "C" void keys(const float* x, int n, uint32_t* out) {
    for (int i = 0; i < n; ++i) out[i] = score_key(x[i]);
}
extern "C" int tests_agree(const float* x, int n, uint32_t lo, uint32_t hi) {
    const RangeTest is = range_test(Range{lo, hi, 0, 0});
    for (int i = 0; i < n; ++i) {
        const uint32_t key = score_key(x[i]);
        const bool over = x[i] >= is.over, in = (is.all || x[i] >= is.floor) && !over;
        if (over != (key > hi) || in != (key >= lo && key <= hi)) return i + 1;
    }
    return 0;
}
// kept[i] = 1 for the `need` that stay; returns marks + 16 narrows, or -1 when the counts are wrong
extern "C" int select_row(const float* x, int n, int need, uint32_t lo, uint32_t hi, int exact,
                          uint8_t* kept) {
    Row row{x, n, need, exact ? Range{0u, 0xffffffffu, 0, n} : Range{lo, hi, 0, 0}, {}, {}};
    const bool listed = settle_range(row, exact != 0);
    const int steps = row.marks + 16 * row.narrows;
    if (listed) {
        for (int pass = 0; pass < kSelPasses && row.g.lo != row.g.hi; ++pass)
            row.narrow_by((int)row.list.size(), [&](int i) { return x[row.list[i]]; });
    }
    if (row.g.lo != row.g.hi) return -1;
    const uint32_t cut = row.g.lo;
    int ties = need - row.g.above;
    if (ties < 1) return -1;
    if (listed) {  // out of the marks and the list
        for (int i = 0; i < n; ++i) kept[i] = (uint8_t)row.above[i];
        for (int i : row.list) kept[i] |= score_key(x[i]) > cut;
        for (int i : row.list)
            if (score_key(x[i]) == cut && ties-- > 0) kept[i] = 1;
    } else {
        for (int i = 0; i < n; ++i) {
            const uint32_t key = score_key(x[i]);
            kept[i] = key > cut || (key == cut && ties-- > 0);
        }
    }
    return steps;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cc = shutil.which("g++")
    assert cc, "g++ is needed to build the host form of the boundary search"
    where = tmp_path_factory.mktemp("select_range")
    src, so = where / "host.cpp", where / "host.so"
    src.write_text(SOURCE)
    subprocess.run([cc, "-O2", "-std=c++17", "-shared", "-fPIC", "-x", "c++", "-I", _build.CSRC,
                    str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(os.fspath(so))
    f, u = ctypes.POINTER(ctypes.c_float), ctypes.c_uint32
    lib.tests_agree.argtypes = [f, ctypes.c_int, u, u]
    lib.select_row.argtypes = [f, ctypes.c_int, ctypes.c_int, u, u, ctypes.c_int,
                               ctypes.POINTER(ctypes.c_uint8)]
    lib.keys.argtypes = [f, ctypes.c_int, ctypes.POINTER(u)]
    return lib


def ptr(x, c):
    return x.ctypes.data_as(ctypes.POINTER(c))


def keys_of(x):
    """NaN 0, else the rank-preserving word of the number, -0 as +0."""
    x = np.where(x == 0, np.float32(0), x).astype(np.float32)
    u = x.view(np.uint32)
    k = np.where(u >> 31 == 1, ~u, u | np.uint32(1 << 31)).astype(np.uint32)
    return np.where(np.isnan(x), np.uint32(0), k).astype(np.uint32)


def kept_of(x, need):
    order = np.lexsort((np.arange(x.size), -keys_of(x).astype(np.int64)))
    out = np.zeros(x.size, dtype=np.uint8)
    out[order[:need]] = 1
    return out


def proposals(x, need, rng):
    """Ranges that a sample may propose: order statistics around the boundary and far from it,
    and the open ends."""
    s = np.sort(keys_of(x[rng.integers(0, x.size, 1024)]))[::-1]
    mean = need / x.size * 1024
    sd = np.sqrt(mean * (1 - need / x.size))
    up, down = mean - 3.5 * sd - 2, mean + 3.5 * sd + 2
    yield (int(s[int(down)]) if down < 1024 else 0, int(s[int(up)]) if up >= 0 else 0xffffffff)
    yield int(s[-1]), int(s[0])          # the whole sample
    yield int(s[0]), int(s[0])           # one key, mostly the wrong one
    yield int(s[-1]), int(s[-1])
    yield 0, 0xffffffff


def check(host, x, need, rng):
    x = np.ascontiguousarray(x, dtype=np.float32)
    want = kept_of(x, need)
    for lo, hi in proposals(x, need, rng):
        for exact in (0, 1):
            if exact and x.size > 2048:
                continue
            got = np.zeros(x.size, dtype=np.uint8)
            steps = host.select_row(ptr(x, ctypes.c_float), x.size, need, lo, hi, exact,
                                    ptr(got, ctypes.c_uint8))
            assert steps >= 0 and steps % 16 <= 2 and steps // 16 <= 3, (steps, hex(lo), hex(hi))
            assert np.array_equal(got, want), (x.size, need, hex(lo), hex(hi), got.sum())


def row(n, rng, **shares):
    """n scores: normal ones, with shares of them replaced."""
    x = rng.standard_normal(n).astype(np.float32)
    at = rng.permutation(n)
    for value, share in shares.items():
        m = int(round(share * n)) if share <= 1 else int(share)
        here, at = at[:m], at[m:]
        if value == "tiny":
            x[here] = rng.choice([-1, 1], m) * rng.integers(0, 5, m) * np.float32(1.4e-45)
        elif value == "zeros":
            x[here] = rng.choice([-0.0, 0.0], m)
        elif value == "lowest":
            x[here] = np.finfo(np.float32).min
        else:
            x[here] = {"nan": np.nan, "low": -np.inf, "high": np.inf}[value]
    return x


def test_compares_stand_for_keys(host):
    """x against range_test is score_key(x) against the range, at and next to every special key."""
    rng = np.random.default_rng(1)
    fmax, tiny = np.finfo(np.float32).max, np.float32(1.4e-45)
    x = np.concatenate([np.float32([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, tiny, -tiny, 1e-38,
                                    -1e-38, 1, -1, fmax, -fmax]), row(300, rng)]).astype(np.float32)
    k = np.zeros(x.size, dtype=np.uint32)
    host.keys(ptr(x, ctypes.c_float), x.size, ptr(k, ctypes.c_uint32))
    assert np.array_equal(k, keys_of(x))
    marks = {0, 1, 0x1fffff, 0x200000, 0x600000, 0x7ffffe, 0x7fffff, 0x800000, 0x7ffffffe, 0x7fffffff,
             0x80000000, 0x80000001, 0xff7fffff, 0xff800000, 0xff800001, 0xffe00000, 0xffffffff}
    marks |= {int(v) for v in k[:20]} | {int(v) - 1 for v in k[:20] if v} | {int(v) + 1 for v in k[:20]}
    for lo in sorted(marks):
        for hi in sorted(marks):
            if lo <= hi:
                at = host.tests_agree(ptr(x, ctypes.c_float), x.size, lo, hi)
                assert at == 0, (hex(lo), hex(hi), x[at - 1])


@pytest.mark.parametrize("n", [300, 2048, 2049, 5000, 20000])
@pytest.mark.parametrize("shares", [
    {}, {"nan": 0.1}, {"nan": 0.6}, {"low": 0.1}, {"low": 0.6}, {"nan": 0.3, "low": 0.3},
    {"high": 0.3, "low": 0.2, "nan": 0.2}, {"zeros": 0.6, "low": 0.015}, {"tiny": 0.9},
    {"tiny": 0.5, "nan": 0.2}, {"lowest": 0.5, "low": 0.2}, {"nan": 1.0}, {"low": 1.0}, {"zeros": 1.0}])
def test_rows_with_odd_scores(host, n, shares):
    rng = np.random.default_rng(n + 7 * len(shares))
    x = row(n, rng, **shares)
    k = keys_of(x)
    edges = {1, 2, n // 2, n - 2, n - 1, int(n * 0.99)}
    for value in (0, 0x7fffff, 0x80000000, 0xff800000):  # both sides of each special value's run
        for edge in (int((k > value).sum()), int((k >= value).sum())):
            edges |= {edge - 1, edge, edge + 1}
    for need in sorted(e for e in edges if 1 <= e < n):
        check(host, x, need, rng)


def test_rows_that_did_not_end(host):
    """-inf, or NaN, at the boundary of long rows, and more of the range than the list holds."""
    for seed in range(2):
        rng = np.random.default_rng(seed)
        check(host, row(300000, rng, low=5000), 300000 - 2500, rng)
        check(host, row(300000, rng, nan=5000), 300000 - 2500, rng)
        check(host, row(20030, rng, low=30, zeros=20000), 20020, rng)
        check(host, row(20000, rng, low=300, zeros=12000), 19800, rng)
        check(host, row(5000, rng, nan=3000), 4000, rng)
