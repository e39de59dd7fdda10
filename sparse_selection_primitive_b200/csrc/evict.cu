// Eviction from a cache by accumulated attention weight: of each row's n keys
// the first `first`, the last `last` and, of the rest, those with the largest
// scores stay, `budget` in all, in the order of their positions.  Entry point:
// lapsum_evict (include/lapsum.h).
//
// Selection: one block per row finds the exact boundary score by radix selection
// over order-preserving integer keys, then walks the row once and writes the kept
// positions in order; equal scores at the boundary go to the lowest positions.
// Gathering: one thread per 16 bytes of a kept row, over all rows at once.
#include <cstdint>
#include <type_traits>

#include "elements.cuh"
#include "lapsum_common.cuh"
#include "lapsum_kernels.h"

namespace lapsum {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

struct EvictArgs {
    int64_t rows;  // B * H
    int H;
    int64_t N, budget, first, last;
    int64_t score_b, score_h;
    const float* score;
    const int32_t* lengths;
};

// NaN sorts below every number (its weight is unknown), -0 as +0.
__device__ __forceinline__ uint32_t score_key(float s) {
    return isnan(s) ? 0u : to_key(s + 0.f);
}

__device__ __forceinline__ int64_t row_length(const EvictArgs& a, int64_t b) {
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n > a.N ? a.N : n;
}

// Exclusive block-wide prefix sum of two counts packed in one word pair.
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

__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(EvictArgs a, int32_t* positions, int32_t* lengths_out) {
    pdl_wait();
    __shared__ unsigned hist[256];
    __shared__ int2 sums[kSelWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int64_t s_need;
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
    const int64_t lo = a.first, hi = n - a.last;  // the keys that compete
    if (threadIdx.x == 0) {
        s_prefix = 0;
        s_need = a.budget - a.first - a.last;
    }
    // the key of the need-th largest competitor, eight bits at a time
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t prefix = s_prefix;
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int64_t i = lo + threadIdx.x; i < hi; i += kSelThreads) {
            const uint32_t key = score_key(score[i]);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int64_t need = s_need;
            int d = 255;
            for (; d > 0 && (int64_t)hist[d] < need; --d) need -= hist[d];
            s_need = need;
            s_prefix = prefix | ((uint32_t)d << shift);
        }
        __syncthreads();
    }
    const uint32_t cut = s_prefix;
    const int64_t ties = s_need;  // how many competitors equal to the cut stay
    int64_t out = 0, tied = 0;
    for (int64_t base = 0; base < n; base += kSelThreads) {
        const int64_t i = base + threadIdx.x;
        bool keep = false, tie = false;
        if (i < n) {
            if (i < lo || i >= hi) keep = true;
            else {
                const uint32_t key = score_key(score[i]);
                keep = key > cut;
                tie = key == cut;
            }
        }
        int2 tot;
        const int2 at = block_prefix(make_int2(keep, tie), &tot, sums);
        // kept so far = kept outright + the ties among the first `ties`
        const int64_t tie_at = tied + at.y;
        const int64_t taken = (tie_at < ties ? tie_at : ties) - (tied < ties ? tied : ties);
        if (keep || (tie && tie_at < ties)) pos[out + at.x + taken] = (int32_t)i;
        const int64_t t2 = tied + tot.y;
        out += tot.x + (t2 < ties ? t2 : ties) - (tied < ties ? tied : ties);
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
        if (p >= 0) {
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
    for (int i = 0; i < 16; ++i)
        if (strides[i] < 0) return LAPSUM_EINVAL;
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
        e = launch_pdl(evict_select_kernel, dim3((unsigned)a.rows), dim3(kSelThreads), 0, st, a,
                       positions, lengths_out);
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
