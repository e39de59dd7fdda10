// Rows of a batch moved to their experts and back.  Entry points:
// lapsum_expert_plan, lapsum_expert_gather, lapsum_expert_combine,
// lapsum_expert_combine_backward (include/lapsum.h).
//
// The plan is a stable counting sort of the T k assignments by expert, with the
// dropped ones (no expert) behind the last expert, so that `slots` is always a
// permutation of 0 .. T k - 1.  Every later step goes by `slots` alone: a row of x is
// read once and written to its k places, and a row of the result is summed from
// its k places in the order j = 0 .. k - 1, so nothing depends on the order in
// which blocks run.
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "elements.cuh"
#include "lapsum_common.cuh"
#include "lapsum_kernels.h"

namespace lapsum {
namespace {

constexpr int kPlanMaxE = 1024;
constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanRounds = 8;                             // of 32 assignments a warp
constexpr int kPlanChunk = kPlanThreads * kPlanRounds;     // assignments per block
constexpr int kPlanFew = 64;  // chunks whose counts every block adds up by itself
constexpr int kExpertMaxK = 32;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ int bucket(const int32_t* experts, int64_t i, int E) {
    const int e = experts[i];
    return (unsigned)e < (unsigned)E ? e : E;
}

// Counts of one chunk's assignments per bucket (E + 1 of them).
__global__ void __launch_bounds__(kPlanThreads)
    plan_count_kernel(const int32_t* experts, int64_t N, int E, int32_t* counts) {
    pdl_wait();
    extern __shared__ int plan_smem[];
    for (int e = threadIdx.x; e <= E; e += kPlanThreads) plan_smem[e] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kPlanChunk;
#pragma unroll
    for (int i = 0; i < kPlanChunk / kPlanThreads; ++i) {
        const int64_t at = base + i * kPlanThreads + threadIdx.x;
        if (at < N) atomicAdd(&plan_smem[bucket(experts, at, E)], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kPlanThreads)
        counts[(int64_t)blockIdx.x * (E + 1) + e] = plan_smem[e];
}

// Many chunks: their counts become each bucket's total of the lower chunks, and the
// totals follow as one more row.  A block takes 32 buckets, a warp 1/32 of the chunks.
__global__ void __launch_bounds__(1024)
    plan_scan_kernel(int32_t* counts, int chunks, int buckets) {
    pdl_wait();
    __shared__ int sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane, per = (chunks + 31) / 32;
    const int c0 = warp * per, c1 = c0 + per < chunks ? c0 + per : chunks;
    int sum = 0;
    if (e < buckets)
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += counts[(int64_t)c * buckets + e];
    sums[warp][lane] = sum;
    __syncthreads();
    int at = 0;
    for (int w = 0; w < warp; ++w) at += sums[w][lane];
    if (e >= buckets) return;
    if (warp == 31) counts[(int64_t)chunks * buckets + e] = at + sum;
    for (int c = c0; c < c1; ++c) {
        const int n = counts[(int64_t)c * buckets + e];
        counts[(int64_t)c * buckets + e] = at;
        at += n;
    }
}

// Places of one chunk's assignments.  A bucket's first place in this chunk is the
// total of the lower buckets plus this bucket's counts in the lower chunks;
// inside the chunk the warps own consecutive runs of assignments and each warp
// walks its run in order, 32 at a time (lanes with the same bucket are ranked by a match).
__global__ void __launch_bounds__(kPlanThreads)
    plan_place_kernel(const int32_t* experts, int64_t N, int E, const int32_t* counts,
                      int chunks, int32_t* offsets, int32_t* slots, int32_t* order) {
    pdl_wait();
    extern __shared__ int plan_smem[];
    const int buckets = E + 1;
    int* total = plan_smem;                  // [buckets] over all chunks
    int* lower = plan_smem + buckets;        // [buckets] over the lower ones
    int* warp_at = plan_smem + 2 * buckets;  // [warps][buckets] the warps' next places
    __shared__ int warp_total[kPlanWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a short chunk is shared out evenly too
    const int64_t start = (int64_t)blockIdx.x * kPlanChunk;
    const int here = (int)(N - start < kPlanChunk ? N - start : kPlanChunk);
    const int rounds = (here + kPlanThreads - 1) / kPlanThreads;
    const int64_t base = start + warp * (rounds * 32);
    int mine[kPlanRounds];
#pragma unroll
    for (int i = 0; i < kPlanRounds; ++i) {
        const int64_t at = base + i * 32 + lane;
        mine[i] = i < rounds && at < N ? bucket(experts, at, E) : -1;
    }
    for (int i = threadIdx.x; i < kPlanWarps * buckets; i += kPlanThreads) warp_at[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPlanRounds; ++i)
        if (mine[i] >= 0) atomicAdd(&warp_at[warp * buckets + mine[i]], 1);
    if (chunks == 1) __syncthreads();
    for (int e = threadIdx.x; e < buckets; e += kPlanThreads) {
        int all = 0, low = 0;
        if (chunks == 1) {
#pragma unroll
            for (int w = 0; w < kPlanWarps; ++w) all += warp_at[w * buckets + e];
        } else if (chunks <= kPlanFew) {
#pragma unroll 8
            for (int c = 0; c < chunks; ++c) {
                const int n = counts[(int64_t)c * buckets + e];
                all += n;
                low += c < (int)blockIdx.x ? n : 0;
            }
        } else {
            all = counts[(int64_t)chunks * buckets + e];
            low = counts[(int64_t)blockIdx.x * buckets + e];
        }
        total[e] = all;
        lower[e] = low;
    }
    __syncthreads();
    // exclusive scan of the totals; each thread owns a run of buckets
    const int per = (buckets + kPlanThreads - 1) / kPlanThreads;
    const int e0 = threadIdx.x * per, e1 = e0 + per < buckets ? e0 + per : buckets;
    int run = 0;
    for (int e = e0; e < e1; ++e) run += total[e];
    int inc = run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) warp_total[warp] = inc;
    __syncthreads();
    int first = inc - run;
    for (int w = 0; w < warp; ++w) first += warp_total[w];
    for (int e = e0; e < e1; ++e) {
        if (blockIdx.x == 0) offsets[e] = first;
        int at = first + lower[e];
        first += total[e];
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            const int n = warp_at[w * buckets + e];
            warp_at[w * buckets + e] = at;
            at += n;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPlanRounds; ++i) {
        if (i >= rounds) break;
        const unsigned same = __match_any_sync(kAll, mine[i]);
        const int64_t at = base + i * 32 + lane;
        int place = 0;
        if (mine[i] >= 0)
            place = warp_at[warp * buckets + mine[i]] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (mine[i] >= 0) {
            if (lane == __ffs(same) - 1) warp_at[warp * buckets + mine[i]] += __popc(same);
            slots[at] = place;
            order[place] = (int32_t)at;
        }
        __syncwarp();
    }
}

// xs[slot(t, j)] = x[t], zeros at the places behind the last expert.  A thread
// moves W elements of a row and writes them k times.
template <class T, int W>
__global__ void __launch_bounds__(256)
    expert_gather_kernel(const T* x, int64_t ld, int64_t T_, int k, int64_t H,
                         const int32_t* slots, const int32_t* live, T* xs) {
    pdl_wait();
    const int64_t cols = H / W, n = T_ * cols;
    const int32_t end = min((int64_t)*live, T_ * k);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = i / cols, c = (i - t * cols) * W;
        const Pack<T, W> v = *reinterpret_cast<const Pack<T, W>*>(x + t * ld + c);
        Pack<T, W> zero;
#pragma unroll
        for (int j = 0; j < W; ++j) zero.v[j] = narrow<T>(0.f);
        for (int j = 0; j < k; ++j) {
            const int32_t s = slots[t * k + j];
            if ((uint64_t)s >= (uint64_t)(T_ * k)) continue;  // no slot of a plan
            *reinterpret_cast<Pack<T, W>*>(xs + (int64_t)s * H + c) = s < end ? v : zero;
        }
    }
}

// out[t] = sum_j w[t, j] y[slot(t, j)] (w null: ones), in fp32 in the order of j,
// rounded once.
template <class T, int W>
__global__ void __launch_bounds__(256)
    expert_combine_kernel(const T* y, int64_t T_, int k, int64_t H, const int32_t* slots,
                          const int32_t* live, const float* w, T* out) {
    pdl_wait();
    const int64_t cols = H / W, n = T_ * cols;
    const int32_t end = min((int64_t)*live, T_ * k);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = i / cols, c = (i - t * cols) * W;
        float acc[W];
#pragma unroll
        for (int q = 0; q < W; ++q) acc[q] = 0.f;
        for (int j = 0; j < k; ++j) {
            const int32_t s = slots[t * k + j];
            if (s < 0 || s >= end) continue;
            const float wj = w != nullptr ? w[t * k + j] : 1.f;
            const Pack<T, W> v = *reinterpret_cast<const Pack<T, W>*>(y + (int64_t)s * H + c);
#pragma unroll
            for (int q = 0; q < W; ++q) acc[q] = fmaf(wj, widen(v.v[q]), acc[q]);
        }
        Pack<T, W> o;
#pragma unroll
        for (int q = 0; q < W; ++q) o.v[q] = narrow<T>(acc[q]);
        *reinterpret_cast<Pack<T, W>*>(out + t * H + c) = o;
    }
}

// dy[slot(t, j)] = w[t, j] dout[t], dw[t, j] = dout[t] . y[slot(t, j)]; zeros for
// the dropped assignments.  One block per row.
template <class T, int W>
__global__ void __launch_bounds__(256)
    expert_combine_backward_kernel(const T* dout, int64_t ld, const T* y, int64_t T_, int k,
                                   int64_t H, const int32_t* slots, const int32_t* live,
                                   const float* w, T* dy, float* dw) {
    pdl_wait();
    __shared__ float part[kExpertMaxK][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t end = min((int64_t)*live, T_ * k);
    const int64_t t = blockIdx.x;
    for (int j = 0; j < k; ++j) {
        const int32_t s = slots[t * k + j];
        if ((uint64_t)s >= (uint64_t)(T_ * k)) {  // no slot of a plan
            if (lane == 0) part[j][warp] = 0.f;
            continue;
        }
        const bool on = s < end;
        const float wj = on ? w[t * k + j] : 0.f;
        float dot = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * W; c < H; c += 256 * W) {
            Pack<T, W> o;
            if (on) {
                const Pack<T, W> g = *reinterpret_cast<const Pack<T, W>*>(dout + t * ld + c);
                const Pack<T, W> v = *reinterpret_cast<const Pack<T, W>*>(y + (int64_t)s * H + c);
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    dot = fmaf(widen(g.v[q]), widen(v.v[q]), dot);
                    o.v[q] = narrow<T>(wj * widen(g.v[q]));
                }
            } else {
#pragma unroll
                for (int q = 0; q < W; ++q) o.v[q] = narrow<T>(0.f);
            }
            *reinterpret_cast<Pack<T, W>*>(dy + (int64_t)s * H + c) = o;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(kAll, dot, d);
        if (lane == 0) part[j][warp] = dot;
    }
    __syncthreads();
    if ((int)threadIdx.x < k) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[threadIdx.x][i];
        dw[t * k + threadIdx.x] = s;
    }
}

// Calls f with the widest pack of elements that all rows allow.
template <class T, class F>
cudaError_t with_pack(size_t align, int64_t H, int64_t ld, F f) {
    const uint64_t bytes = (uint64_t)align | (uint64_t)(H * (int64_t)sizeof(T)) |
                           (uint64_t)(ld * (int64_t)sizeof(T)) | 16u;
    const int a = (int)(bytes & (~bytes + 1));  // the largest power of two that divides all
    if (a >= 16) return f(std::integral_constant<int, 16 / (int)sizeof(T)>{});
    if (a == 8) return f(std::integral_constant<int, 8 / (int)sizeof(T)>{});
    if constexpr (sizeof(T) == 2)
        if (a == 4) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1>{});
}

unsigned stream_grid(int64_t work) {
    const int64_t most = (int64_t)device_sm_count() * 16, want = (work + 255) / 256;
    return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}

bool rows_ok(int64_t T, int32_t k, int64_t H) {
    return T >= 1 && k >= 1 && k <= kExpertMaxK && H >= 1 && T <= (int64_t(1) << 31) - 1 &&
           T * k < (int64_t(1) << 31);
}

size_t address_bits(const void* p) { return reinterpret_cast<size_t>(p); }

}  // namespace
}  // namespace lapsum

using namespace lapsum;

extern "C" size_t lapsum_expert_plan_workspace_bytes(int64_t N, int64_t E) {
    if (N < 1 || N >= (int64_t(1) << 31) || E < 1 || E > kPlanMaxE) return 0;
    const int64_t chunks = (N + kPlanChunk - 1) / kPlanChunk;
    const size_t need = chunks > 1 ? (size_t)(chunks + 1) * (size_t)(E + 1) * 4 : 0;
    return (need + 255) / 256 * 256 + 256;
}

extern "C" int lapsum_expert_plan(const int32_t* experts, int64_t N, int64_t E, int32_t* offsets,
                                  int32_t* slots, int32_t* order, void* ws, size_t ws_bytes,
                                  void* stream) {
    if (experts == nullptr || offsets == nullptr || slots == nullptr || order == nullptr)
        return LAPSUM_EINVAL;
    const size_t need = lapsum_expert_plan_workspace_bytes(N, E);
    if (need == 0) return LAPSUM_EINVAL;
    if (!aligned_to(experts, 4) || !aligned_to(offsets, 4) || !aligned_to(slots, 4) ||
        !aligned_to(order, 4))
        return LAPSUM_EINVAL;
    if (ws == nullptr || !aligned_to(ws, 256) || ws_bytes < need) return LAPSUM_EWORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    const int chunks = (int)((N + kPlanChunk - 1) / kPlanChunk);
    int32_t* counts = (int32_t*)ws;
    ProfScope prof("expert_plan", st);
    if (chunks > 1) {
        const cudaError_t e =
            launch_pdl(plan_count_kernel, dim3(chunks), dim3(kPlanThreads), (size_t)(E + 1) * 4, st,
                       experts, N, (int)E, counts);
        if (e != cudaSuccess) return LAPSUM_ECUDA;
    }
    if (chunks > kPlanFew) {
        const cudaError_t e = launch_pdl(plan_scan_kernel, dim3((unsigned)(E + 32) / 32), dim3(1024),
                                         0, st, counts, chunks, (int)E + 1);
        if (e != cudaSuccess) return LAPSUM_ECUDA;
    }
    static std::atomic<unsigned long long> done{0};
    once_per_device(done, [] {
        cudaFuncSetAttribute(plan_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (kPlanWarps + 2) * (kPlanMaxE + 1) * 4);
    });
    const cudaError_t e = launch_pdl(
        plan_place_kernel, dim3(chunks), dim3(kPlanThreads),
        (size_t)(kPlanWarps + 2) * (E + 1) * 4, st, experts, N, (int)E, (const int32_t*)counts, chunks,
        offsets, slots, order);
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}

extern "C" int lapsum_expert_gather(const void* x, int dtype, int64_t ld, int64_t T, int32_t k,
                                    int64_t H, const int32_t* slots, const int32_t* live, void* xs,
                                    void* stream) {
    if (x == nullptr || slots == nullptr || live == nullptr || xs == nullptr) return LAPSUM_EINVAL;
    if (!known_dtype(dtype) || !rows_ok(T, k, H) || ld < H) return LAPSUM_EINVAL;
    const int size = dtype_size(dtype);
    if (!aligned_to(x, size) || !aligned_to(xs, size) || !aligned_to(slots, 4) ||
        !aligned_to(live, 4))
        return LAPSUM_EINVAL;
    cudaStream_t st = (cudaStream_t)stream;
    ProfScope prof("expert_gather", st);
    const cudaError_t e = with_dtype(dtype, [&](auto* tag) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        return with_pack<E>(address_bits(x) | address_bits(xs), H, ld, [&](auto w) {
            constexpr int W = decltype(w)::value;
            return launch_pdl(expert_gather_kernel<E, W>, dim3(stream_grid(T * (H / W))),
                              dim3(256), 0, st, (const E*)x, ld, T, (int)k, H, slots, live, (E*)xs);
        });
    });
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}

extern "C" int lapsum_expert_combine(const void* y, int dtype, int64_t T, int32_t k, int64_t H,
                                     const int32_t* slots, const int32_t* live,
                                     const float* weights, void* out, void* stream) {
    if (y == nullptr || slots == nullptr || live == nullptr || out == nullptr) return LAPSUM_EINVAL;
    if (!known_dtype(dtype) || !rows_ok(T, k, H)) return LAPSUM_EINVAL;
    const int size = dtype_size(dtype);
    if (!aligned_to(y, size) || !aligned_to(out, size) || !aligned_to(slots, 4) ||
        !aligned_to(live, 4) || !aligned_to(weights, 4))
        return LAPSUM_EINVAL;
    cudaStream_t st = (cudaStream_t)stream;
    ProfScope prof("expert_combine", st);
    const cudaError_t e = with_dtype(dtype, [&](auto* tag) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        return with_pack<E>(address_bits(y) | address_bits(out), H, H, [&](auto w) {
            constexpr int W = decltype(w)::value;
            return launch_pdl(expert_combine_kernel<E, W>, dim3(stream_grid(T * (H / W))),
                              dim3(256), 0, st, (const E*)y, T, (int)k, H, slots, live, weights,
                              (E*)out);
        });
    });
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}

extern "C" int lapsum_expert_combine_backward(const void* dout, int dtype, int64_t ld,
                                              const void* y, int64_t T, int32_t k, int64_t H,
                                              const int32_t* slots, const int32_t* live,
                                              const float* weights, void* dy, float* dweights,
                                              void* stream) {
    if (dout == nullptr || y == nullptr || slots == nullptr || live == nullptr ||
        weights == nullptr || dy == nullptr || dweights == nullptr)
        return LAPSUM_EINVAL;
    if (!known_dtype(dtype) || !rows_ok(T, k, H) || ld < H) return LAPSUM_EINVAL;
    const int size = dtype_size(dtype);
    if (!aligned_to(dout, size) || !aligned_to(y, size) || !aligned_to(dy, size) ||
        !aligned_to(slots, 4) || !aligned_to(live, 4) || !aligned_to(weights, 4) ||
        !aligned_to(dweights, 4))
        return LAPSUM_EINVAL;
    cudaStream_t st = (cudaStream_t)stream;
    ProfScope prof("expert_combine_backward", st);
    const cudaError_t e = with_dtype(dtype, [&](auto* tag) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        return with_pack<E>(address_bits(dout) | address_bits(y) | address_bits(dy), H, ld,
                            [&](auto w) {
                                constexpr int W = decltype(w)::value;
                                return launch_pdl(expert_combine_backward_kernel<E, W>,
                                                  dim3((unsigned)T), dim3(256), 0, st,
                                                  (const E*)dout, ld, (const E*)y, T, (int)k, H,
                                                  slots, live, weights, (E*)dy, dweights);
                            });
    });
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}
