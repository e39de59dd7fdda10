// The boundary search of the eviction, without anything of CUDA's own, so that a host
// test can run the same steps: keys of scores, the float compares that stand for compares
// of keys, and the order of the steps, which ends after a fixed number of them.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

#ifdef __CUDACC__
#define LAPSUM_BOTH __host__ __device__ __forceinline__
#else
#define LAPSUM_BOTH inline
#endif

namespace lapsum {

constexpr int kSelBits = 11, kSelBins = 1 << kSelBits;
constexpr int kSelList = 8192;
// A histogram pass cuts a range of 32 bits to 21, 10 and 0 bits (one key).
constexpr int kSelPasses = 3;

// NaN sorts below every number (its weight is unknown), -0 as +0.
LAPSUM_BOTH uint32_t score_key(float s) {
    const float x = s + 0.f;
    uint32_t u;
    memcpy(&u, &x, 4);
    if (x != x) return 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The least number whose key is `key` or more; a NaN where there is none.  Keys below that
// of -inf belong to no number (0 is the key of every NaN): read as a float they are NaN, with
// which every compare is false.  The same holds past +inf.
LAPSUM_BOTH float number_from(uint32_t key) {
    if (key < 0x007fffffu) return -INFINITY;
    const uint32_t u = (key & 0x80000000u) ? (key & 0x7fffffffu) : ~key;
    float x;
    memcpy(&x, &u, 4);
    return x;
}

// What the boundary is known to lie in: it is the need-th largest key of the competitors,
// `above` of them have keys above hi and `inside` keys in [lo, hi].
struct Range {
    uint32_t lo, hi;
    int above, inside;
};

// The same as compares of the scores: key(x) > hi is x >= over (-0 >= +0, and both have the
// key of +0), and key(x) >= lo is x >= floor, or anything at all for lo = 0.
struct RangeTest {
    float floor, over;
    bool all;
};
LAPSUM_BOTH RangeTest range_test(Range g) {
    return RangeTest{number_from(g.lo), number_from(g.hi < 0xff800000u ? g.hi + 1u : g.hi | 0xff800001u),
                     g.lo == 0u};
}

// By how much a key's distance from lo is shifted to give its bin: at most kSelBins bins.
LAPSUM_BOTH int range_shift(uint32_t lo, uint32_t hi) {
#ifdef __CUDA_ARCH__
    const int bits = 32 - __clz(hi - lo);
#else
    const int bits = hi == lo ? 0 : 32 - __builtin_clz(hi - lo);
#endif
    return bits > kSelBits ? bits - kSelBits : 0;
}

// The range of one bin, which holds the boundary: `above` of the keys lie above the bin,
// `inside` in it.
LAPSUM_BOTH Range range_of_bin(Range g, int bin, int above, int inside) {
    const int shift = range_shift(g.lo, g.hi);
    const uint32_t lo = g.lo + ((uint32_t)bin << shift);
    const uint64_t hi = (uint64_t)lo + (1ull << shift) - 1;
    return Range{lo, hi < g.hi ? (uint32_t)hi : g.hi, above, inside};
}

// The steps, after which the list holds the keys of row.range() (true), or the range is the
// boundary's one key (false).  row.mark() marks the keys above the range and lists those in
// it, and returns the counts; row.narrow() makes the range the boundary's bin of it, with
// counts.  `exact`: the range at the start is certain (else sampled, its counts unknown).
template <class Row>
LAPSUM_BOTH bool settle_range(Row& row, bool exact) {
    if (!exact) {
        const Range g = row.mark();
        if (g.above < row.need && row.need - g.above <= g.inside) {
            row.set(g);
            if (g.inside <= kSelList) return true;
        } else {  // the sample missed
            row.set(Range{0u, 0xffffffffu, 0, row.competitors});
        }
    }
    for (int pass = 0; pass <= kSelPasses; ++pass) {
        const Range g = row.range();
        if (g.lo == g.hi) return false;
        if (g.inside <= kSelList) {
            row.mark();
            return true;
        }
        row.narrow();
    }
    return false;
}

}  // namespace lapsum
