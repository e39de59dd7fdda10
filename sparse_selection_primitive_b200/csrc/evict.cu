// Eviction from a cache by accumulated attention weight: of each row's n keys
// the first `first`, the last `last` and, of the rest, those with the largest
// scores stay, `budget` in all, in the order of their positions.  Entry point:
// lapsum_evict (include/lapsum.h).
//
// Selection, one block per row.  Scores become order-preserving integer keys.  A
// sample of the row gives a range [lo, hi] of keys that holds the boundary key with
// high probability (the bracketing of section 2.2 of the pages, on order statistics
// of plain samples); one pass over the row then marks the keys above the range in a bit map
// and lists those inside, and the boundary is found in the list by radix selection.
// Counts prove the range right; where they do not, or where the list would
// overflow, histogram passes over the row narrow the range first, three at most
// (select_range.cuh).  The kept positions come out of the bit map in order, so nothing is
// sorted; keys equal to the boundary have a bit map of their own, of which the first
// (lowest positions) are taken.
// Gathering: one thread per 16 bytes of a kept row, over all rows at once.
//
// 256 x 65536 (lengths from a quarter of that) to 1024: selection 35 us (7 us of bytes), of
// which the sample takes about 5, the pass 10 to 18 (108 of 148 SMs hold two rows), the list 5
// and the bit maps 3; four histogram passes and block-wide prefixes took 211.  Bringing the row
// into L2 while the sample is sorted made it 2 us slower.  Gathering 26.5 us (20.8 us of bytes);
// several rows a thread (more loads in flight, fewer threads) made it 36 to 52.
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "bitonic.cuh"
#include "elements.cuh"
#include "lapsum_common.cuh"
#include "lapsum_kernels.h"
#include "select_range.cuh"

namespace lapsum {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelSample = 2 * kSelThreads;
constexpr int64_t kSelWindow = int64_t(1) << 18;  // positions that the bit maps hold at a time
static_assert(kSelSample <= kSelList, "the sample is sorted where the list will stand");
constexpr unsigned kAll = 0xffffffffu;

struct EvictArgs {
    int64_t rows;  // B * H
    int H;
    int64_t N, budget, first, last;
    int64_t score_b, score_h;
    const float* score;
    const int32_t* lengths;
};

__device__ __forceinline__ int64_t row_length(const EvictArgs& a, int64_t b) {
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n > a.N ? a.N : n;
}

// Exclusive block-wide prefix sum of a pair of counts; *tot gets the totals.
__device__ __forceinline__ int2 block_prefix(int2 v, int2* tot, int2* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(kAll, inc.x, d), y = __shfl_up_sync(kAll, inc.y, d);
        if (lane >= d) {
            inc.x += x;
            inc.y += y;
        }
    }
    __syncthreads();
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int2 before = make_int2(0, 0), all = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
        const int2 s = sums[w];
        if (w < warp) {
            before.x += s.x;
            before.y += s.y;
        }
        all.x += s.x;
        all.y += s.y;
    }
    *tot = all;
    return make_int2(before.x + inc.x - v.x, before.y + inc.y - v.y);
}

struct SelShared {
    alignas(16) unsigned hist[kSelBins];
    int2 sums[kSelWarps];
    Range range;
    int listed;               // keys listed (may exceed the room)
    int above;
};

// Adds one to a bin; a warp whose active lanes all want the same bin adds once.
__device__ __forceinline__ void count_bin(unsigned* hist, int bin) {
    const unsigned on = __activemask();
    int same;
    __match_all_sync(on, bin, &same);
    if (same) {
        if ((threadIdx.x & 31) == __ffs(on) - 1) atomicAdd(&hist[bin], (unsigned)__popc(on));
    } else {
        atomicAdd(&hist[bin], 1u);
    }
}

// Narrows the range to the bin that holds the need-th largest key.  The histogram of
// the keys inside the range is complete; every thread calls.
__device__ void narrow_range(SelShared& sh, int need) {
    __syncthreads();
    const Range g = sh.range;
    // thread t owns four neighbouring bins, the highest ones first
    static_assert(kSelBins == 4 * kSelThreads, "four bins a thread");
    const int bin0 = kSelBins - 4 - 4 * (int)threadIdx.x;
    const uint4 q = *reinterpret_cast<const uint4*>(&sh.hist[bin0]);
    const int c[4] = {(int)q.w, (int)q.z, (int)q.y, (int)q.x};
    int2 tot;
    int at = g.above + block_prefix(make_int2(c[0] + c[1] + c[2] + c[3], 0), &tot, sh.sums).x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (at < need && need <= at + c[i]) sh.range = range_of_bin(g, bin0 + 3 - i, at, c[i]);
        at += c[i];
    }
    __syncthreads();
}

__device__ __forceinline__ void clear_words(uint32_t* w, int64_t n) {
    for (int64_t i = threadIdx.x; i < n; i += kSelThreads) w[i] = 0;
}

// Calls f(position, key) for this thread's share of the positions [lo, hi), which is four
// consecutive ones at a time.
template <class F>
__device__ __forceinline__ void each_key(const float* score, int64_t lo, int64_t hi, F f) {
    // up to the first 16-byte boundary and from the last on, one at a time
    const int64_t skew = (int64_t)((reinterpret_cast<uintptr_t>(score + lo) & 15u) / 4);
    int64_t head = lo + (skew ? 4 - skew : 0);
    if (head > hi) head = hi;
    const int64_t quads = (hi - head) / 4, tail = head + quads * 4;
    if (threadIdx.x < head - lo) f(lo + threadIdx.x, score_key(score[lo + threadIdx.x]));
    if (threadIdx.x < hi - tail) f(tail + threadIdx.x, score_key(score[tail + threadIdx.x]));
    const float4* s4 = reinterpret_cast<const float4*>(score + head);
    constexpr int kUnroll = 4;
    int64_t i = threadIdx.x;
    for (; i + (kUnroll - 1) * kSelThreads < quads; i += kUnroll * kSelThreads) {
        float4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = __ldg(s4 + i + u * kSelThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t at = head + (i + u * kSelThreads) * 4;
            f(at, score_key(v[u].x));
            f(at + 1, score_key(v[u].y));
            f(at + 2, score_key(v[u].z));
            f(at + 3, score_key(v[u].w));
        }
    }
    for (; i < quads; i += kSelThreads) {
        const float4 v = __ldg(s4 + i);
        const int64_t at = head + i * 4;
        f(at, score_key(v.x));
        f(at + 1, score_key(v.y));
        f(at + 2, score_key(v.z));
        f(at + 3, score_key(v.w));
    }
}

// A sample of the competitors brackets the boundary: two keys a thread, sorted across
// the block, and the order statistics 3.5 standard deviations either side of the expected
// rank.  `sorted` holds kSelSample words.
__device__ void sample_range(SelShared& sh, uint32_t* sorted, const float* score, int64_t lo,
                             int64_t hi, int64_t need) {
    const int64_t n = hi - lo;
    // four neighbours (one memory sector, mostly) from each of kSelSample / 4 equal
    // stretches; two threads share them
    const int stretch = threadIdx.x >> 1;
    uint32_t x = (uint32_t)stretch * 0x9e3779b9u;
    x ^= x >> 15;
    x *= 0x85ebca6bu;
    x ^= x >> 13;
    const int64_t a = n * stretch / (kSelSample / 4), b = n * (stretch + 1) / (kSelSample / 4);
    const float* at = score + lo + a + (int64_t)(x % (uint32_t)(b - a - 3)) + (threadIdx.x & 1) * 2;
    uint32_t v[2] = {score_key(at[0]), score_key(at[1])};
    bitonic_sort_row<2, kSelThreads, kSelThreads>(v, threadIdx.x, sorted);
    sorted[kSelSample - 1 - 2 * threadIdx.x] = v[0];  // descending
    sorted[kSelSample - 2 - 2 * threadIdx.x] = v[1];
    __syncthreads();
    if (threadIdx.x == 0) {
        const double q = (double)need / (double)n, mean = q * kSelSample;
        const double sd = sqrt(mean * (1.0 - q));
        const double up = mean - 3.5 * sd - 2.0, down = mean + 3.5 * sd + 2.0;
        sh.range = Range{down < kSelSample ? sorted[(int)down] : 0u,
                         up >= 0.0 ? sorted[(int)up] : 0xffffffffu, 0, 0};
    }
    __syncthreads();
}

// The marking pass over the competitors [lo, hi): bits of `above` for the keys above
// g.hi (not when it is null), and the positions of the keys in [g.lo, g.hi] listed as far
// as the list has room; sh.above and sh.listed count them.  A thread compares four runs
// of four positions with the range, as floats (range_test), while the next four are on their
// way; its warp makes room for all its finds with one addition.
__device__ void mark_and_list(SelShared& sh, const float* score, int64_t lo, int64_t hi, Range g,
                              uint32_t* above, int32_t* list_at) {
    constexpr int kRuns = 4;
    const int lane = threadIdx.x & 31;
    const RangeTest is = range_test(g);
    unsigned over = 0;
    // at: position of v[0].x, the runs `step` positions apart; use: bit 4 u + j for each
    // value that counts
    auto take = [&](int64_t at, int step, const float4 (&v)[kRuns], unsigned use) {
        unsigned in = 0, top = 0;
#pragma unroll
        for (int u = 0; u < kRuns; ++u) {
            const float x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (x[j] >= is.floor) in |= 1u << (4 * u + j);
                if (x[j] >= is.over) top |= 1u << (4 * u + j);
            }
        }
        if (is.all) in = 0xffffu;
        in &= use & ~top;
        top &= use;
        over += __popc(top);
        if (above != nullptr)
            while (top) {
                const int k = __ffs(top) - 1;
                top &= top - 1;
                const int p = (int)at + (k >> 2) * step + (k & 3);
                atomicOr(&above[p >> 5], 1u << (p & 31));
            }
        if (!__any_sync(kAll, in)) return;
        const int mine = __popc(in);
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(kAll, inc, d);
            if (lane >= d) inc += o;
        }
        int base = 0;
        if (lane == 31) base = atomicAdd(&sh.listed, inc);
        base = __shfl_sync(kAll, base, 31) + inc - mine;
        while (in) {
            const int k = __ffs(in) - 1;
            in &= in - 1;
            if (base < kSelList) list_at[base] = (int)at + (k >> 2) * step + (k & 3);
            ++base;
        }
        __syncwarp();
    };
    const int64_t skew = (int64_t)((reinterpret_cast<uintptr_t>(score + lo) & 15u) / 4);
    int64_t head = lo + (skew ? 4 - skew : 0);
    if (head > hi) head = hi;
    const int64_t quads = (hi - head) / 4, tail = head + quads * 4;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    if (threadIdx.x < 32) {  // up to the first 16-byte boundary, and from the last on
        const int64_t at = lane < 4 ? lo + lane : tail + lane - 4;
        const bool on = lane < 4 ? at < head : lane < 8 && at < hi;
        const float4 v[kRuns] = {make_float4(on ? score[at] : 0.f, 0.f, 0.f, 0.f), zero, zero, zero};
        take(at, 0, v, on ? 1u : 0u);
    }
    const float4* s4 = reinterpret_cast<const float4*>(score + head);
    auto load = [&](int64_t base, float4 (&x)[kRuns]) {
#pragma unroll
        for (int u = 0; u < kRuns; ++u) {
            const int64_t i = base + u * kSelThreads + lane;
            x[u] = i < quads ? __ldg(s4 + i) : zero;
        }
    };
    float4 x[kRuns];
    int64_t base = (int)threadIdx.x - lane;
    load(base, x);
    for (; base < quads; base += kRuns * kSelThreads) {
        float4 next[kRuns];
        load(base + kRuns * kSelThreads, next);
        unsigned use = 0;
#pragma unroll
        for (int u = 0; u < kRuns; ++u)
            if (base + u * kSelThreads + lane < quads) use |= 15u << (4 * u);
        take(head + (base + lane) * 4, 4 * kSelThreads, x, use);
#pragma unroll
        for (int u = 0; u < kRuns; ++u) x[u] = next[u];
    }
    if (over) atomicAdd(&sh.above, (int)over);
}

// The steps of settle_range on one row; every thread calls them.
struct BoundarySearch {
    SelShared& sh;
    const float* score;
    int64_t lo, hi;
    int need, competitors;
    int64_t words;        // of a bit map of the row
    uint32_t *above_map;  // null: the row is longer than the bit maps
    uint32_t* tie_map;
    int32_t* list_at;

    __device__ __forceinline__ Range range() const { return sh.range; }
    __device__ __forceinline__ void set(Range g) {
        __syncthreads();
        if (threadIdx.x == 0) sh.range = g;
        __syncthreads();
    }
    __device__ __forceinline__ Range mark() {
        __syncthreads();
        if (threadIdx.x == 0) {
            sh.listed = 0;
            sh.above = 0;
        }
        if (above_map != nullptr) {
            clear_words(above_map, words);
            clear_words(tie_map, words);
        }
        __syncthreads();
        const Range g = sh.range;
        mark_and_list(sh, score, lo, hi, g, above_map, list_at);
        __syncthreads();
        return Range{g.lo, g.hi, sh.above, sh.listed};
    }
    __device__ __forceinline__ void narrow() {
        __syncthreads();
        clear_words(sh.hist, kSelBins);
        __syncthreads();
        const Range g = sh.range;
        const int shift = range_shift(g.lo, g.hi);
        each_key(score, lo, hi, [&](int64_t, uint32_t key) {
            if (key >= g.lo && key <= g.hi) count_bin(sh.hist, (int)((key - g.lo) >> shift));
        });
        narrow_range(sh, need);
    }
};

__global__ void __launch_bounds__(kSelThreads, 2)
    evict_select_kernel(EvictArgs a, int64_t window, int32_t* positions, int32_t* lengths_out) {
    pdl_wait();
    extern __shared__ uint32_t sel_smem[];
    __shared__ SelShared sh;
    uint32_t* list_key = sel_smem;                  // [kSelList]
    int32_t* list_at = (int32_t*)(sel_smem + kSelList);
    uint32_t* above_map = sel_smem + 2 * kSelList;  // a bit per position of a window
    uint32_t* tie_map = above_map + window / 32;
    const int64_t r = blockIdx.x, b = r / a.H, h = r - b * a.H;
    const int64_t n = row_length(a, b);
    const float* score = a.score + b * a.score_b + h * a.score_h;
    int32_t* pos = positions + r * a.budget;
    const int64_t kept = n < a.budget ? n : a.budget;
    if (h == 0 && threadIdx.x == 0) lengths_out[b] = (int32_t)kept;
    for (int64_t i = kept + threadIdx.x; i < a.budget; i += kSelThreads) pos[i] = -1;
    if (n <= a.budget) {
        for (int64_t i = threadIdx.x; i < n; i += kSelThreads) pos[i] = (int32_t)i;
        return;
    }
    const int64_t lo = a.first, hi = n - a.last;  // the positions that compete
    const int need = (int)(a.budget - a.first - a.last);
    const bool one = n <= window;                 // the whole row fits the bit maps
    bool marked = false;                          // they are filled
    if (need > 0) {
        if (hi - lo <= 2 * kSelSample) {
            if (threadIdx.x == 0) sh.range = Range{0u, 0xffffffffu, 0, (int)(hi - lo)};
            __syncthreads();
        } else {
            sample_range(sh, list_key, score, lo, hi, need);
        }
        BoundarySearch search{sh,    score, lo,   hi,        need, (int)(hi - lo), (n + 31) / 32,
                              one ? above_map : nullptr, tie_map, list_at};
        const bool listed = settle_range(search, hi - lo <= 2 * kSelSample);
        if (listed) {
            const int m = sh.listed < kSelList ? sh.listed : kSelList;
            for (int i = threadIdx.x; i < m; i += kSelThreads) list_key[i] = score_key(score[list_at[i]]);
            for (int pass = 0; pass < kSelPasses && sh.range.lo != sh.range.hi; ++pass) {
                const Range g = sh.range;
                __syncthreads();
                clear_words(sh.hist, kSelBins);
                __syncthreads();
                const int shift = range_shift(g.lo, g.hi);
                for (int i = threadIdx.x; i < m; i += kSelThreads) {
                    const uint32_t key = list_key[i];
                    if (key >= g.lo && key <= g.hi) atomicAdd(&sh.hist[(key - g.lo) >> shift], 1u);
                }
                narrow_range(sh, need);
            }
            if (one) {
                const uint32_t cut = sh.range.lo;
                for (int i = threadIdx.x; i < m; i += kSelThreads) {
                    const uint32_t key = list_key[i];
                    const int32_t at = list_at[i];
                    if (key > cut) atomicOr(&above_map[at >> 5], 1u << (at & 31));
                    if (key == cut) atomicOr(&tie_map[at >> 5], 1u << (at & 31));
                }
                marked = true;
            }
        }
    }
    __syncthreads();
    const uint32_t cut = need > 0 ? sh.range.lo : 0xffffffffu;
    const int64_t ties = need > 0 ? need - sh.range.above : 0;  // competitors at the cut that stay
    // the first and the last stay whatever their scores
    for (int64_t i = threadIdx.x; i < a.first; i += kSelThreads) pos[i] = (int32_t)i;
    for (int64_t i = threadIdx.x; i < a.last; i += kSelThreads)
        pos[a.budget - a.last + i] = (int32_t)(hi + i);
    // the competitors out of the bit maps, a window of positions at a time; nothing is stored
    // past their room, not even when the scores change meanwhile
    const int64_t room = a.budget - a.last;
    int64_t out = a.first, tied = 0;
    for (int64_t w0 = 0; w0 < n; w0 += window) {
        const int64_t w1 = w0 + window < n ? w0 + window : n;
        const int words = (int)((w1 - w0 + 31) / 32);
        if (!marked) {
            __syncthreads();
            clear_words(above_map, words);
            clear_words(tie_map, words);
            __syncthreads();
            if (need > 0)
                each_key(score, lo < w0 ? w0 : lo < w1 ? lo : w1, hi < w0 ? w0 : hi < w1 ? hi : w1,
                         [&](int64_t at, uint32_t key) {
                             const int i = (int)(at - w0);
                             if (key > cut) atomicOr(&above_map[i >> 5], 1u << (i & 31));
                             if (key == cut) atomicOr(&tie_map[i >> 5], 1u << (i & 31));
                         });
            __syncthreads();
        }
        // each thread owns a run of words: its kept competitors come after those of lower
        // threads; of the ties only the first `ties` of the row count
        const int per = (words + kSelThreads - 1) / kSelThreads;
        const int i0 = threadIdx.x * per, i1 = i0 + per < words ? i0 + per : words;
        int2 mine = make_int2(0, 0);
        for (int i = i0; i < i1; ++i) {
            mine.x += __popc(above_map[i]);
            mine.y += __popc(tie_map[i]);
        }
        int2 tot;
        const int2 at = block_prefix(mine, &tot, sh.sums);
        const int64_t was = tied < ties ? tied : ties;
        const int64_t t0 = tied + at.y;
        int64_t o = out + at.x + ((t0 < ties ? t0 : ties) - was);
        int64_t left = ties - t0;
        for (int i = i0; i < i1; ++i) {
            const uint32_t T = tie_map[i];
            uint32_t bits = above_map[i] | T;
            while (bits) {
                const int k = __ffs(bits) - 1;
                bits &= bits - 1;
                if (((T >> k) & 1u) && left-- <= 0) continue;
                if (o < room) pos[o] = (int32_t)(w0 + (int64_t)i * 32 + k);
                ++o;
            }
        }
        const int64_t t2 = tied + tot.y;
        out += tot.x + ((t2 < ties ? t2 : ties) - was);
        tied = t2;
    }
}

struct GatherArgs {
    int64_t kb, kh, kr, vb, vh, vr;        // element strides of the caches read
    int64_t okb, okh, okr, ovb, ovh, ovr;  // of the caches written
    int64_t osb, osh;                      // of the scores written
};

template <class T, int W>
__global__ void __launch_bounds__(256)
    evict_gather_kernel(EvictArgs a, GatherArgs g, int D, const int32_t* positions, const T* k,
                        const T* v, T* k_out, T* v_out, float* score_out) {
    pdl_wait();
    const int cols = D / W;
    const int64_t n = a.rows * a.budget * cols;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / cols;
        const int c = (int)(i - row * cols) * W;
        const int64_t r = row / a.budget, j = row - r * a.budget, b = r / a.H, h = r - b * a.H;
        const int64_t p = positions[row];
        Pack<T, W> kk, vv;
        float s = 0.f;
        if (p >= 0 && p < a.N) {  // a place left open by scores that change meanwhile is no position
            kk = *reinterpret_cast<const Pack<T, W>*>(k + b * g.kb + h * g.kh + p * g.kr + c);
            vv = *reinterpret_cast<const Pack<T, W>*>(v + b * g.vb + h * g.vh + p * g.vr + c);
            if (c == 0) s = a.score[b * a.score_b + h * a.score_h + p];
        } else {
#pragma unroll
            for (int q = 0; q < W; ++q) kk.v[q] = vv.v[q] = narrow<T>(0.f);
        }
        *reinterpret_cast<Pack<T, W>*>(k_out + b * g.okb + h * g.okh + j * g.okr + c) = kk;
        *reinterpret_cast<Pack<T, W>*>(v_out + b * g.ovb + h * g.ovh + j * g.ovr + c) = vv;
        if (c == 0) score_out[b * g.osb + h * g.osh + j] = s;
    }
}

}  // namespace
}  // namespace lapsum

using namespace lapsum;

extern "C" int lapsum_evict(const void* k, const void* v, int dtype, const float* score,
                            const int32_t* lengths, const int64_t* strides, int64_t B, int64_t H,
                            int64_t N, int64_t D, int64_t budget, int64_t first, int64_t last,
                            void* k_out, void* v_out, float* score_out, int32_t* positions,
                            int32_t* lengths_out, void* stream) {
    if (k == nullptr || v == nullptr || score == nullptr || lengths == nullptr ||
        strides == nullptr || k_out == nullptr || v_out == nullptr || score_out == nullptr ||
        positions == nullptr || lengths_out == nullptr)
        return LAPSUM_EINVAL;
    const int64_t big = int64_t(1) << 31;
    if (!known_dtype(dtype) || B < 1 || H < 1 || N < 1 || D < 1 || B >= big || H >= big ||
        N >= big || D > 65536 || B * H >= big)
        return LAPSUM_EINVAL;
    if (budget < 1 || budget >= big || first < 0 || last < 0 || first > budget ||
        last > budget - first)
        return LAPSUM_EINVAL;
    // the stride of a dimension of one element means nothing
    const int64_t extent[16] = {B, H, N, B, H, N, B, H, B, H, budget, B, H, budget, B, H};
    int64_t own[16];
    for (int i = 0; i < 16; ++i) {
        own[i] = extent[i] > 1 ? strides[i] : 0;
        if (own[i] < 0) return LAPSUM_EINVAL;
    }
    strides = own;
    const int size = dtype_size(dtype);
    if (!aligned_to(k, size) || !aligned_to(v, size) || !aligned_to(k_out, size) ||
        !aligned_to(v_out, size) || !aligned_to(score, 4) || !aligned_to(score_out, 4) ||
        !aligned_to(lengths, 4) || !aligned_to(positions, 4) || !aligned_to(lengths_out, 4))
        return LAPSUM_EINVAL;
    EvictArgs a{B * H, (int)H, N, budget, first, last, strides[6], strides[7], score, lengths};
    GatherArgs g{strides[0], strides[1], strides[2], strides[3], strides[4],  strides[5],
                 strides[8], strides[9], strides[10], strides[11], strides[12], strides[13],
                 strides[14], strides[15]};
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    {
        ProfScope prof("evict_select", st);
        static std::atomic<unsigned long long> done{0};
        const int64_t window = N < kSelWindow ? (N + 31) / 32 * 32 : kSelWindow;
        once_per_device(done, [] {
            cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(kSelList * 8 + kSelWindow / 4));
        });
        e = launch_pdl(evict_select_kernel, dim3((unsigned)a.rows), dim3(kSelThreads),
                       (size_t)(kSelList * 8 + window / 4), st, a, window, positions, lengths_out);
    }
    if (e != cudaSuccess) return LAPSUM_ECUDA;
    ProfScope prof("evict_gather", st);
    // the widest pack that every row start and length allows
    uint64_t bits = (uint64_t)(uintptr_t)k | (uint64_t)(uintptr_t)v | (uint64_t)(uintptr_t)k_out |
                    (uint64_t)(uintptr_t)v_out | (uint64_t)(D * size) | 16u;
    for (int i = 0; i < 14; ++i)
        if (i != 6 && i != 7) bits |= (uint64_t)(strides[i] * size);
    const int align = (int)(bits & (~bits + 1));
    e = with_dtype(dtype, [&](auto* tag) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        auto go = [&](auto w) {
            constexpr int W = decltype(w)::value;
            const int64_t work = a.rows * budget * (D / W), want = (work + 255) / 256,
                          most = (int64_t)device_sm_count() * 16;
            return launch_pdl(evict_gather_kernel<T, W>, dim3((unsigned)(want < most ? want : most)),
                              dim3(256), 0, st, a, g, (int)D, (const int32_t*)positions,
                              (const T*)k, (const T*)v, (T*)k_out, (T*)v_out, score_out);
        };
        if (align >= 16) return go(std::integral_constant<int, 16 / (int)sizeof(T)>{});
        if (align == 8) return go(std::integral_constant<int, 8 / (int)sizeof(T)>{});
        return go(std::integral_constant<int, 1>{});
    });
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}
