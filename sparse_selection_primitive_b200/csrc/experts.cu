// Rows of a batch moved to their experts and back.  Entry points:
// lapsum_expert_plan, lapsum_expert_gather, lapsum_expert_combine,
// lapsum_expert_combine_backward, lapsum_expert_combine_backward_part (include/lapsum.h).
//
// The plan is a stable counting sort of the T k assignments by expert, with the
// dropped ones (no expert) behind the last expert, so that `slots` is always a
// permutation of 0 .. T k - 1.  Every later step goes by `slots` alone: a row of x is
// read once and written to its k places, and a row of the result is summed from
// its k places in the order j = 0 .. k - 1, so nothing depends on the order in
// which blocks run.
//
// The rows are bound by DRAM: 16384 x 8 rows of 4 KB, gather 96 us (94 us of bytes at the copy
// rate), combine 101 (94), backward of the combination 192 (177).  The plan of 131072
// assignments takes 19 us in two launches, that of 512 takes 6 in one: chains of dependent
// steps, with next to nothing to read.
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

// The row kernels: a block of kRowThreads threads takes kRowThreads / TX rows at a time, TX
// threads (a power of two, enough for a row or all of the block) to each, so that no
// thread divides to find its place.  A thread moves 16 bytes of a row at a time: one pack of W
// elements where all rows are aligned for it, else U shorter packs TX apart.  More loads in
// flight a thread (several assignments at once) took the combination of 16384 x 8 rows of 4 KB
// from 100 to 126-144 us: fewer threads fit, and rows are long enough to fill the memory pipe.
constexpr int kRowThreads = 256;

struct RowArgs {
    int64_t ld, T, H, N;  // N = T k
    int k, tx;            // tx: log2 of TX
    const int32_t* slots;
    const int32_t* live;
};

__device__ __forceinline__ int64_t own_row(const RowArgs& a) {
    return (int64_t)blockIdx.x * (kRowThreads >> a.tx) + (threadIdx.x >> a.tx);
}
__device__ __forceinline__ int64_t row_step(const RowArgs& a) {
    return (int64_t)gridDim.x * (kRowThreads >> a.tx);
}
__device__ __forceinline__ int32_t live_rows(const RowArgs& a) {
    const int64_t n = *a.live;
    return (int32_t)(n < a.N ? n : a.N);
}
template <class T, int W>
constexpr int packs_of() {
    return 16 / (W * (int)sizeof(T));
}
// The U packs of a row from column c on, `step` columns apart, as far as the row goes.
template <class T, int W, int U>
__device__ __forceinline__ void load_packs(const T* row, int64_t c, int step, int64_t H,
                                           Pack<T, W> (&v)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (U == 1 || c + u * step < H)
            v[u] = *reinterpret_cast<const Pack<T, W>*>(row + c + u * step);
}
template <class T, int W, int U>
__device__ __forceinline__ void store_packs(T* row, int64_t c, int step, int64_t H,
                                            const Pack<T, W> (&v)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (U == 1 || c + u * step < H) *reinterpret_cast<Pack<T, W>*>(row + c + u * step) = v[u];
}

// xs[slot(t, j)] = x[t], zeros at the places behind the last expert.
template <class T, int W>
__global__ void __launch_bounds__(kRowThreads)
    expert_gather_kernel(RowArgs a, const T* x, T* xs) {
    constexpr int U = packs_of<T, W>();
    pdl_wait();
    const int64_t t = own_row(a);
    if (t >= a.T) return;
    const int32_t end = live_rows(a);
    const int TX = 1 << a.tx, step = TX * W;
    for (int64_t c = (int64_t)(threadIdx.x & (TX - 1)) * W; c < a.H; c += U * step) {
        Pack<T, W> v[U], zero[U];
        load_packs<T, W, U>(x + t * a.ld, c, step, a.H, v);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < W; ++q) zero[u].v[q] = narrow<T>(0.f);
        for (int j = 0; j < a.k; ++j) {
            const int32_t s = a.slots[t * a.k + j];
            if (s < 0 || s >= a.N) continue;  // no slot of a plan
            if (s < end) store_packs<T, W, U>(xs + (int64_t)s * a.H, c, step, a.H, v);
            else store_packs<T, W, U>(xs + (int64_t)s * a.H, c, step, a.H, zero);
        }
    }
}

// out[t] = sum_j w[t, j] y[slot(t, j)] (w null: ones), in fp32 in the order of j,
// rounded once.
template <class T, int W>
__global__ void __launch_bounds__(kRowThreads, 8)
    expert_combine_kernel(RowArgs a, const T* y, const float* w, T* out) {
    constexpr int U = packs_of<T, W>();
    pdl_wait();
    const int32_t end = live_rows(a);
    const int TX = 1 << a.tx, step = TX * W;
    for (int64_t t = own_row(a); t < a.T; t += row_step(a))
        for (int64_t c = (int64_t)(threadIdx.x & (TX - 1)) * W; c < a.H; c += U * step) {
            float acc[U * W];
#pragma unroll
            for (int q = 0; q < U * W; ++q) acc[q] = 0.f;
            for (int j = 0; j < a.k; ++j) {
                const int32_t s = a.slots[t * a.k + j];
                if (s < 0 || s >= end) continue;
                const float wj = w != nullptr ? w[t * a.k + j] : 1.f;
                Pack<T, W> v[U];
                load_packs<T, W, U>(y + (int64_t)s * a.H, c, step, a.H, v);
#pragma unroll
                for (int q = 0; q < U * W; ++q)
                    acc[q] = fmaf(wj, widen(v[q / W].v[q % W]), acc[q]);
            }
            Pack<T, W> o[U];
#pragma unroll
            for (int q = 0; q < U * W; ++q) o[q / W].v[q % W] = narrow<T>(acc[q]);
            store_packs<T, W, U>(out + t * a.H, c, step, a.H, o);
        }
}

// dy[slot(t, j)] = w[t, j] dout[t], dw[t, j] = dout[t] . y[slot(t, j)]; zeros for the
// dropped assignments.  TX is 32 at least, so that whole warps share a row's products, and
// known to the compiler, which then unrolls the walk along the row: 197 us instead of 247 for
// 16384 x 8 rows of 4 KB, 189 instead of 388 for rows of 2049 16-bit elements (half as many).
// kDy, kDw: which of the two is formed; without dw y is not read.
template <class T, int W, int TX, bool kDy, bool kDw>
__global__ void __launch_bounds__(kRowThreads)
    expert_combine_backward_kernel(RowArgs a, const T* dout, const T* y, const float* w, T* dy,
                                   float* dw) {
    pdl_wait();
    __shared__ float part[kRowThreads / 32][kExpertMaxK];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = threadIdx.x % TX;
    const int64_t t = (int64_t)blockIdx.x * (kRowThreads / TX) + threadIdx.x / TX;
    if (t < a.T) {
        const int32_t end = live_rows(a);
        for (int j = 0; j < a.k; ++j) {
            const int32_t s = a.slots[t * a.k + j];
            float dot = 0.f;
            if (s >= 0 && s < a.N) {  // else no slot of a plan
                const bool on = s < end;
                const float wj = on ? w[t * a.k + j] : 0.f;
                for (int64_t c = at * W; c < a.H; c += TX * W) {
                    Pack<T, W> o;
                    if (on) {
                        const Pack<T, W> g = *reinterpret_cast<const Pack<T, W>*>(dout + t * a.ld + c);
                        Pack<T, W> v;
                        if constexpr (kDw) v = *reinterpret_cast<const Pack<T, W>*>(y + (int64_t)s * a.H + c);
#pragma unroll
                        for (int q = 0; q < W; ++q) {
                            if constexpr (kDw) dot = fmaf(widen(g.v[q]), widen(v.v[q]), dot);
                            o.v[q] = narrow<T>(wj * widen(g.v[q]));
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < W; ++q) o.v[q] = narrow<T>(0.f);
                    }
                    if constexpr (kDy) *reinterpret_cast<Pack<T, W>*>(dy + (int64_t)s * a.H + c) = o;
                }
            }
            if constexpr (kDw) {
#pragma unroll
                for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(kAll, dot, d);
                if (lane == 0) part[warp][j] = dot;
            }
        }
    }
    if constexpr (!kDw) return;
    __syncthreads();
    if (t < a.T && at < a.k) {  // thread j of a row adds up its warps' parts
        const int w0 = threadIdx.x / TX * (TX / 32);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < TX / 32; ++i) s += part[w0 + i][at];
        dw[t * a.k + at] = s;
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

// Threads that a row of H elements keeps busy at 16 bytes each.
template <class T, int W>
int64_t row_threads(int64_t H) {
    return (H / W + packs_of<T, W>() - 1) / packs_of<T, W>();
}
// Threads to a row: `threads`, up to a power of two, `least` at least.
RowArgs row_args(int64_t ld, int64_t T, int32_t k, int64_t H, const int32_t* slots,
                 const int32_t* live, int64_t threads, int least) {
    RowArgs a{ld, T, H, T * k, (int)k, 0, slots, live};
    while ((1 << a.tx) < kRowThreads && ((1 << a.tx) < threads || (1 << a.tx) < least)) ++a.tx;
    return a;
}
// Blocks that take every row once (at most T < 2^31 of them), or, for kernels that walk on by
// row_step, as many as stay busy.
int64_t row_blocks(const RowArgs& a) {
    const int64_t rows = kRowThreads >> a.tx;
    return (a.T + rows - 1) / rows;
}
dim3 row_grid(const RowArgs& a) { return dim3((unsigned)row_blocks(a)); }
dim3 walking_row_grid(const RowArgs& a) {
    const int64_t want = row_blocks(a), most = (int64_t)device_sm_count() * 16;
    return dim3((unsigned)(want < most ? want : most));
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
            const RowArgs a = row_args(ld, T, k, H, slots, live, row_threads<E, W>(H), 1);
            return launch_pdl(expert_gather_kernel<E, W>, row_grid(a), dim3(kRowThreads), 0, st, a,
                              (const E*)x, (E*)xs);
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
            const RowArgs a = row_args(H, T, k, H, slots, live, row_threads<E, W>(H), 1);
            return launch_pdl(expert_combine_kernel<E, W>, walking_row_grid(a), dim3(kRowThreads), 0, st, a,
                              (const E*)y, weights, (E*)out);
        });
    });
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}

namespace {

int combine_backward(const void* dout, int dtype, int64_t ld, const void* y, int64_t T, int32_t k,
                     int64_t H, const int32_t* slots, const int32_t* live, const float* weights,
                     void* dy, float* dweights, void* stream) {
    if (dout == nullptr || slots == nullptr || live == nullptr || weights == nullptr ||
        (y == nullptr && dweights != nullptr) || (dy == nullptr && dweights == nullptr))
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
        return with_pack<E>(address_bits(dout) | address_bits(y) | address_bits(dy), H, ld, [&](auto w) {
            constexpr int W = decltype(w)::value;
            const RowArgs a = row_args(ld, T, k, H, slots, live, H / W, 32);
            const auto go = [&](auto tx) {
                constexpr int TX = decltype(tx)::value;
                const auto run = [&](auto kernel) {
                    return launch_pdl(kernel, row_grid(a), dim3(kRowThreads), 0, st, a, (const E*)dout,
                                      (const E*)y, weights, (E*)dy, dweights);
                };
                if (dweights == nullptr) return run(expert_combine_backward_kernel<E, W, TX, true, false>);
                if (dy == nullptr) return run(expert_combine_backward_kernel<E, W, TX, false, true>);
                return run(expert_combine_backward_kernel<E, W, TX, true, true>);
            };
            switch (a.tx) {
                case 5: return go(std::integral_constant<int, 32>{});
                case 6: return go(std::integral_constant<int, 64>{});
                case 7: return go(std::integral_constant<int, 128>{});
                default: return go(std::integral_constant<int, 256>{});
            }
        });
    });
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}

}  // namespace

extern "C" int lapsum_expert_combine_backward(const void* dout, int dtype, int64_t ld,
                                              const void* y, int64_t T, int32_t k, int64_t H,
                                              const int32_t* slots, const int32_t* live,
                                              const float* weights, void* dy, float* dweights,
                                              void* stream) {
    if (y == nullptr || dy == nullptr || dweights == nullptr) return LAPSUM_EINVAL;
    return combine_backward(dout, dtype, ld, y, T, k, H, slots, live, weights, dy, dweights, stream);
}

extern "C" int lapsum_expert_combine_backward_part(const void* dout, int dtype, int64_t ld,
                                                   const void* y, int64_t T, int32_t k, int64_t H,
                                                   const int32_t* slots, const int32_t* live,
                                                   const float* weights, void* dy, float* dweights,
                                                   void* stream) {
    return combine_backward(dout, dtype, ld, y, T, k, H, slots, live, weights, dy, dweights, stream);
}
