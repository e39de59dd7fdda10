// Attention over a cache that also accumulates, per key, the weight that the
// queries gave it.  Entry point: lapsum_attend_accumulate (include/lapsum.h).
//
// For each sequence b, key/value head h and query row r = i G + g (token i, and g of the
// G = Hq / Hkv query heads that share h):
//     x_j = scale q_r . k_j  over the keys the row sees,  p = softmax(x),
//     out_r = sum_j p_j v_j,   score[b, h, j] += sum_r p_{r, j}.
//
// Keys take the M side of the matrix instruction: S^T = K Q^T is 128 keys x RT rows, so
// that a few query rows (one token and its G heads) fill a whole instruction, each
// thread holds one key's logits for all rows, and the column sums that the scores need are
// sums inside a thread.  O^T = V^T P is D x RT, with V read as it lies.  Weights go to
// the second product as pairs of 16-bit values, p = hi + lo, which keep 15 bits of p and more
// (Pair says how small a weight may be).  Runs of key tiles are joined by a second kernel;
// scores come from kept logits where few rows share a key, and from a second S^T where
// keeping them would cost more.
// More than kKeepRows rows a key fill the M side themselves (attend_wide_kernel).
//
// 32 x 8192 keys x 8 heads of 128, 8 rows a key: 179 us at full length (169 us of bytes), DRAM
// bound.  2 x 32768 x 8, 128 rows: 72 us for the outputs (42 us of bytes, 21 of products), 35 for
// the scores.  Matrix instructions issued from a branch on the lane number, not by an elected
// thread, cost 15 us of the one and 8 of the other.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "elements.cuh"
#include "lapsum_common.cuh"
#include "lapsum_kernels.h"
#include "tensor_core.cuh"

namespace lapsum {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kTile = 128;          // keys per tile: the M of S^T
constexpr int kKeepRows = 16;       // logits of more rows a key are formed again, not kept
constexpr int kMaxStages = 6;
constexpr int kSms = 148;           // of a B200; plans are made without asking the device
constexpr int kMostRuns = 2 * kSms; // runs of a head: two blocks for each SM
constexpr int kBlockSmem = 223;     // KB of dynamic shared memory of a block that has an SM to itself
constexpr int kJoinThreads = 256, kJoinKeys = 1024;

struct AttendArgs {
    int64_t qb, qh, qr;  // element strides of q: batch, head, token
    int64_t sib, sih, sob, soh;
    int64_t N, R;        // rows per key/value head: Sq * G
    int B, Sq, Hkv, D, G;
    int kh, kb, vh, vb;  // 1 where the caches' head and batch coordinates count, else 0
    float scale_log2;    // scale * log2(e): logits and weights are kept in powers of two
    const int32_t* lengths;
};

// How the work is cut; a function of the sizes alone.
struct AttendPlan {
    int rt;         // rows per tile
    int row_tiles;
    int splits;     // runs of key tiles per row tile
    int stages, smem;
    int keep;       // the logits are kept for the scores
    int64_t RP;     // rows of logits per key, padded
    size_t off_lse, off_part, off_logits, bytes;
};

constexpr int kNarrowThreads = 64 + 128;  // the kernel for up to kKeepRows rows a key, and its
constexpr int kNarrowCols = 128;          // columns of tensor memory: 6 x 16, up to a power of two
constexpr int kWideThreads = 64 + 256;    // the kernel for more
// The score pass over keys whose logits were not kept.
constexpr int kScoreRows = 128, kScoreThreads = 64 + 256;
struct ScorePlan {
    int blocks;  // blocks of a key/value head
    int stages, smem;
};

__device__ __forceinline__ int64_t cache_length(const AttendArgs& a, int64_t b) {
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n > a.N ? a.N : n;
}

// v[i] of all 32 lanes joined, N values: afterwards lane l holds the results of
// N / 32 (or 1) values from index joined_at<N>(l) on.  Each step halves the values a lane
// still holds, so the whole costs about N exchanges instead of 5 N.
template <int N>
__device__ __forceinline__ int joined_at(int lane) {
    int at = 0, half = N / 2;
#pragma unroll
    for (int d = 16; d; d >>= 1)
        if (half >= 1) {
            at += (lane & d) ? half : 0;
            half >>= 1;
        }
    return at;
}
template <int N, class F>
__device__ __forceinline__ void join_lanes(float (&v)[N], int lane, F f) {
    int n = N;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = lane & d;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = f(keep, __shfl_xor_sync(kAll, give, d));
                }
        } else {
            v[0] = f(v[0], __shfl_xor_sync(kAll, v[0], d));
        }
    }
}

template <int N>
__device__ __forceinline__ void softmax_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// A tile of RT rows of q from row0 on into shared memory, zero beyond the rows and beyond
// D, in the layout that TMA gives the keys (128-byte rows, 16-byte chunks exchanged by row).
template <class T, int RT>
__device__ __forceinline__ void load_rows(const AttendArgs& a, const T* q, int b, int h,
                                          int64_t row0, int rows, uint32_t to, int thread,
                                          int threads) {
    // eight chunks (one column block of a row) after another; all of a thread's loads before its
    // stores, which took the start of a block of 128 rows from 12000 cycles to 6500
    constexpr int kBatch = 8;
    const uint32_t total = (a.D + 63) / 64 * (RT * 8);
    for (uint32_t base = thread; base < total; base += threads * kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t i = base + u * threads, r = (i >> 3) % RT, c = i / (RT * 8) * 8 + (i & 7);
            x[u] = make_uint4(0, 0, 0, 0);
            if (i < total && r < (uint32_t)rows && c * 8 < (uint32_t)a.D) {
                const uint32_t row = (uint32_t)row0 + r, tok = row / (uint32_t)a.G,
                               g = row - tok * (uint32_t)a.G;
                x[u] = *reinterpret_cast<const uint4*>(q + b * a.qb + tok * a.qr +
                                                       ((int64_t)h * a.G + g) * a.qh + c * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t i = base + u * threads, r = (i >> 3) % RT, c = i & 7;
            if (i >= total) continue;
            const uint32_t at = to + i / (RT * 8) * (RT * 128) + r * 128 + ((c ^ (r & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[u].x), "r"(x[u].y),
                         "r"(x[u].z), "r"(x[u].w)
                         : "memory");
        }
    }
}

// S^T = K Q^T of one tile (or S = Q K^T, with the operands exchanged): D / 16 steps along
// the rows of both operands, whose 128-byte column blocks lie a tile of keys, or RT rows,
// apart.  The steps only add to the operands' descriptors.
template <int RT>
__device__ __forceinline__ void key_products(uint32_t to, uint64_t k, uint64_t q, int D,
                                             uint32_t shape) {
    for (int sub = 0; sub * 64 < D; ++sub) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            if (sub * 64 + kk * 16 < D)
                mma_f16(to, k + advance(kk * 32), q + advance(kk * 32), shape, sub + kk > 0);
        k += advance(kTile * 128);
        q += advance(RT * 128);
    }
}

// Two weights as words of two 16-bit values each: p = hi + lo / apart, where `apart` is
// kApart if the products of hi and lo are summed apart, else 1.
//
// A weight is 2^(x - m) for a reference m that keeps the row's largest weight between 2^kLift
// and 2^kMost.  The bounds of fp16 make the difference.  Its smallest value is 2^-24, and what
// is below half of that is lost: with lo as it is, up to 2^-25 of a weight, which is 2^-36 of
// the row's largest one; with lo scaled by kApart, 2^-37 and 2^-48.  A reference at the largest
// weight itself, with lo as it is, lost all weights below 2^-25 of the largest from the output
// but not from the sum; with one key that takes nearly all of the weight and has a value near
// 0, that is most of the output.  2^kMost is half of fp16's largest value, and hi leaves lo at
// most 2^(kMost - 12), which kApart takes there too.  bf16 has fp32's range.
template <class T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    static constexpr bool bf16 = true;
    static constexpr float kLift = 0.f, kMost = 12.f, kApart = 1.f;
    // hi is cut off (a byte permutation; conversions run at a quarter of the rate), which
    // leaves lo up to 2^-7 of the weight; lo is rounded: off by 2^-15 of it at most
    static __device__ __forceinline__ void split(float a, float b, float, uint32_t* hi, uint32_t* lo) {
        const uint32_t u = __float_as_uint(a), v = __float_as_uint(b);
        *hi = __byte_perm(u, v, 0x7632);
        const __nv_bfloat162 l =
            __floats2bfloat162_rn(a - __uint_as_float(u & 0xffff0000u), b - __uint_as_float(v & 0xffff0000u));
        *lo = *reinterpret_cast<const uint32_t*>(&l);
    }
};
template <>
struct Pair<__half> {
    static constexpr bool bf16 = false;
    static constexpr float kLift = 11.f, kMost = 15.f, kApart = 4096.f;
    static __device__ __forceinline__ void split(float a, float b, float apart, uint32_t* hi, uint32_t* lo) {
        const __half2 h = __floats2half2_rn(a, b);
        const __half2 l = __floats2half2_rn((a - __low2float(h)) * apart, (b - __high2float(h)) * apart);
        *hi = *reinterpret_cast<const uint32_t*>(&h);
        *lo = *reinterpret_cast<const uint32_t*>(&l);
    }
};

// One run of key tiles for one tile of rows.  Writes the rows' references and sums
// (stats), the unnormalised outputs (part) and, where they are kept, the logits, all in
// fp32.  Warp 0 loads, warp 1 multiplies, and four warps do the softmax, each on the
// quarter of the lanes of tensor memory that it can read.
//
// Weights are 2^(x - m) with a reference m per row, kLift below the exact maximum of the first
// tile, that is raised only when some logit passes it by kMost: a maximum over the keys is a
// maximum across threads, dear to form for every tile, and any reference within a factor
// 2^(kMost - kLift) serves as well.  Raising it rescales the sums and the outputs in tensor
// memory.
template <class T>
__global__ void __launch_bounds__(kNarrowThreads, 2)
    attend_narrow_kernel(AttendArgs a, AttendPlan p, const T* q,
                        const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map, float2* stats, float* part,
                        float* logits) {
    constexpr int RT = kKeepRows;
    constexpr float kLift = Pair<T>::kLift, kMost = Pair<T>::kMost, kApart = Pair<T>::kApart;
    extern __shared__ char smem_raw[];
    __shared__ uint64_t bars[2 * kMaxStages + 4];
    __shared__ uint32_t s_tmem;
    __shared__ int s_failed;
    __shared__ float red[4][RT];
    // per row: the reference (0 while no key was seen), by how much it rose last and what that
    // multiplied sums with; and how far a logit may pass it
    __shared__ alignas(16) float s_ref[RT], s_up[RT], s_scale[RT];
    __shared__ bool s_seen[RT];
    __shared__ float s_slack;
    __shared__ alignas(16) int s_lim[RT];  // keys that each row sees, from the run's first
    const int lane = threadIdx.x & 31, warp = uniform((int)threadIdx.x >> 5);
    const int rt = blockIdx.x % p.row_tiles;
    const int64_t rest = blockIdx.x / p.row_tiles;
    const int split = (int)(rest % p.splits);
    const int64_t bh = rest / p.splits;
    const int b = (int)(bh / a.Hkv), h = (int)(bh % a.Hkv);
    const int64_t row0 = (int64_t)rt * RT;
    const int rows = (int)(a.R - row0 < RT ? a.R - row0 : RT);
    float2* my_stats = stats + (bh * p.splits + split) * a.R + row0;

    pdl_wait();
    const int64_t n = uniform(cache_length(a, b));
    // keys that the tile's last row sees, and this run's tiles among them
    int64_t seen = n - a.Sq + 1 + (row0 + rows - 1) / a.G;
    seen = seen < 0 ? 0 : seen;
    const int64_t all_tiles = (seen + kTile - 1) / kTile;
    const int64_t per = (all_tiles + p.splits - 1) / p.splits;
    const int64_t first = split * per;
    const int tiles = (int)(all_tiles - first < per ? all_tiles - first : per);
    if (tiles <= 0) {
        if (threadIdx.x < rows) my_stats[threadIdx.x] = make_float2(-INFINITY, 0.f);
        return;
    }

    const int subs = (a.D + 63) / 64;                   // 128-byte column blocks of a row
    const uint32_t sub_bytes = kTile * 128, stage_bytes = subs * sub_bytes;
    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t q_at = ring + p.stages * stage_bytes;
    const uint32_t p_at = q_at + subs * RT * 128;       // hi, then lo
    const uint32_t full = smem_addr(bars), empty = full + 8 * kMaxStages,
                   s_done = empty + 8 * kMaxStages, p_full = s_done + 16, p_empty = p_full + 8;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        mbar_init(s_done, 1);
        mbar_init(s_done + 8, 1);
        mbar_init(p_full, 128);
        mbar_init(p_empty, 1);
        fence_barrier_init();
        s_failed = 0;
    }
    if (threadIdx.x < RT) {
        const int most = tiles * kTile;
        int64_t lim = n - a.Sq + 1 + (row0 + threadIdx.x) / a.G - first * kTile;
        lim = lim < 0 ? 0 : lim;
        s_ref[threadIdx.x] = 0.f;
        s_seen[threadIdx.x] = false;
        if (threadIdx.x == 0) s_slack = -INFINITY;
        s_lim[threadIdx.x] = (int)(threadIdx.x < rows && lim < most ? lim : most);
    }
    if (warp == 1) tmem_alloc(smem_addr(&s_tmem), kNarrowCols);
    load_rows<T, RT>(a, q, b, h, row0, rows, q_at, threadIdx.x, kNarrowThreads);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // logits of two tiles, then the outputs of the weights' hi and lo parts
    const uint32_t tmem = uniform(s_tmem), o_col = tmem + 2 * RT;
    // the ring's items: K0, K1, V0, K2, V1, ..., V(last)
    const int items = 2 * tiles;
    auto key_item = [](int t) { return t == 0 ? 0 : 2 * t - 1; };
    auto value_item = [&](int t) { return t + 1 < tiles ? 2 * t + 2 : 2 * t + 1; };
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (; issued < items; ++issued) {
                const int s = issued % p.stages, turn = issued / p.stages;
                if (turn > 0) ok = mbar_wait(empty + 8 * s, (turn - 1) & 1);
                if (!ok) break;
                mbar_expect(full + 8 * s, stage_bytes);
                const bool key = issued == 0 || (issued % 2 == 1 && issued < items - 1);
                const int t = key ? (issued + 1) / 2 : (issued - 1) / 2;
                const int y = (int)((first + t) * kTile);
                for (int c = 0; c < subs; ++c)
                    tma_load_4d(ring + s * stage_bytes + c * sub_bytes, key ? &k_map : &v_map,
                                full + 8 * s, c * 64, y, h * (key ? a.kh : a.vh),
                                b * (key ? a.kb : a.vb));
            }
            if (!ok)  // gave up: let the copies in flight land before the block ends
                for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
                    mbar_wait(full + 8 * (i % p.stages), (i / p.stages) & 1);
        }
    } else if (warp == 1) {
        const uint32_t shape_s = mma_shape(Pair<T>::bf16, false, false, kTile, RT);
        const uint32_t shape_o = mma_shape(Pair<T>::bf16, true, true, 128, 2 * RT);
        const uint64_t q_op = operand(q_at, 16, 1024, kSwizzle128);
        const uint64_t p_op = operand(p_at, 128, 2048, kNoSwizzle);
        auto logits_of = [&](int t) {  // S^T of tile t into its half
            const int item = key_item(t), s = item % p.stages;
            if (!__all_sync(kAll, mbar_wait(full + 8 * s, (item / p.stages) & 1))) return false;
            tc_fence_after();
            if (elect_one()) {
                key_products<RT>(tmem + (t & 1) * RT,
                                 operand(ring + s * stage_bytes, 16, 1024, kSwizzle128), q_op,
                                 a.D, shape_s);
                mma_commit(empty + 8 * s);
                mma_commit(s_done + 8 * (t & 1));
            }
            __syncwarp();
            return true;
        };
        ok = logits_of(0) && (tiles == 1 || logits_of(1));
        for (int t = 0; t < tiles && ok; ++t) {
            const int item = value_item(t), s = item % p.stages;
            ok = mbar_wait(full + 8 * s, (item / p.stages) & 1) && mbar_wait(p_full, t & 1);
            ok = __all_sync(kAll, ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                for (int m = 0; m * 128 < a.D; ++m) {
                    const uint64_t v = operand(ring + s * stage_bytes + m * 2 * sub_bytes, sub_bytes,
                                               1024, kSwizzle128);
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_f16(o_col + m * 2 * RT, v + advance(kk * 2048), p_op + advance(kk * 256),
                                shape_o, t + kk > 0);
                }
                mma_commit(empty + 8 * s);
                mma_commit(p_empty);
            }
            __syncwarp();
            // the softmax has read tile t's half
            if (t + 2 < tiles) ok = logits_of(t + 2);
        }
    } else {
        const int quarter = warp & 3;                  // the lanes of tensor memory it may read
        const int key = quarter * 32 + lane;           // of a tile
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const int own = joined_at<RT>(lane);
        float sum[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) sum[r] = 0.f;
        for (int t = 0; t < tiles; ++t) {
            ok = ok && mbar_wait(s_done + 8 * (t & 1), (t >> 1) & 1);
            ok = __all_sync(kAll, ok);
            tc_fence_after();
            float x[RT];
            tmem_ld<RT>(lanes + (t & 1) * RT, x);
            const int64_t j0 = (first + t) * kTile, j = j0 + key;
#pragma unroll
            for (int r = 0; r < RT; ++r) x[r] *= a.scale_log2;
            if ((t + 1) * kTile > s_lim[0]) {  // the first row sees the fewest
                const int at = t * kTile + key;
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    if (at >= s_lim[r]) x[r] = -INFINITY;
            }
            if (j < n) {
                // the rows of zeros past the last one have NaN where a key is infinite: 0 there
                float* to = logits + (bh * a.N + j) * p.RP + row0;
#pragma unroll
                for (int r = 0; r < RT; r += 4)
                    if (row0 + r < p.RP)
                        *reinterpret_cast<float4*>(to + r) =
                            make_float4(x[r], r + 1 < rows ? x[r + 1] : 0.f, r + 2 < rows ? x[r + 2] : 0.f,
                                        r + 3 < rows ? x[r + 3] : 0.f);
            }
            float over[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                x[r] -= s_ref[r];
                over[r & 3] = fmaxf(over[r & 3], x[r]);
            }
            const bool past = fmaxf(fmaxf(over[0], over[1]), fmaxf(over[2], over[3])) > s_slack;
            // one answer for the four warps
            uint32_t raise;
            asm volatile(
                "{\n\t.reg .pred u, v;\n\tsetp.ne.u32 u, %1, 0;\n\t"
                "barrier.cta.red.or.pred v, 2, 128, u;\n\tselp.u32 %0, 1, 0, v;\n\t}"
                : "=r"(raise)
                : "r"(past ? 1u : 0u)
                : "memory");
            // the outputs so far are complete, and the weights' room is free
            ok = ok && (t == 0 || mbar_wait(p_empty, (t - 1) & 1));
            ok = __all_sync(kAll, ok);
            if (raise) {
                tc_fence_after();
                {
                    float top[RT];
#pragma unroll
                    for (int r = 0; r < RT; ++r) top[r] = x[r];
                    join_lanes<RT>(top, lane, [](float u, float w) { return fmaxf(u, w); });
                    red[quarter][own] = top[0];
                }
                softmax_sync<128>();
                if (key < 32) {
                    bool unseen = false;
                    if (key < RT) {
                        const float by = fmaxf(fmaxf(red[0][key], red[1][key]), fmaxf(red[2][key], red[3][key]));
                        unseen = !s_seen[key] && by == -INFINITY;
                        const float up = unseen ? 0.f : s_seen[key] ? fmaxf(by - kLift, 0.f) : by - kLift;
                        s_ref[key] += up;
                        s_up[key] = up;
                        s_scale[key] = s_seen[key] ? ex2_ftz(-up) : 0.f;
                        s_seen[key] = !unseen;
                    }
                    unseen = __any_sync(kAll, unseen);
                    if (key == 0) s_slack = unseen ? -INFINITY : kMost;
                }
                softmax_sync<128>();
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    x[r] -= s_up[r];
                    sum[r] *= s_scale[r];
                }
                if (t > 0)  // hi and lo parts of the outputs, of the first and the second 128 columns
                    for (int m = 0; m < (a.D + 127) / 128 * 2; ++m) {
                        float o[RT];
                        tmem_ld<RT>(lanes + (2 + m) * RT, o);
#pragma unroll
                        for (int r = 0; r < RT; ++r) o[r] *= s_scale[r];
                        tmem_st<RT>(lanes + (2 + m) * RT, o);
                    }
            }
            if (j0 + kTile > n) {
                // value rows behind the cache's end may hold anything: 0 x NaN is NaN
                const int item = value_item(t), s = item % p.stages;
                ok = ok && mbar_wait(full + 8 * s, (item / p.stages) & 1);
                if (ok && j >= n)
                    for (int c = 0; c < subs * 8; ++c)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         ring + s * stage_bytes + (c >> 3) * sub_bytes + key * 128 +
                                         (c & 7) * 16),
                                     "r"(0)
                                     : "memory");
                __syncwarp();
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                x[r] = ex2_ftz(x[r]);
                sum[r] += x[r];
            }
#pragma unroll
            for (int r = 0; r < RT; r += 8) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    Pair<T>::split(x[r + 2 * i], x[r + 2 * i + 1], kApart, &hi[i], &lo[i]);
                const uint32_t to = p_at + (r >> 3) * 2048 + key * 16;
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(hi[0]),
                             "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
                             : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + RT * 256),
                             "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3])
                             : "memory");
            }
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(p_full);
        }
        join_lanes<RT>(sum, lane, [](float u, float w) { return u + w; });
        if (ok) ok = mbar_wait(p_empty, (tiles - 1) & 1);
        if (!ok) s_failed = 1;
        red[quarter][own] = sum[0];
        softmax_sync<128>();
        tc_fence_after();
        const int tid = threadIdx.x - 64;
        if (tid < rows) {
            const float l = red[0][tid] + red[1][tid] + red[2][tid] + red[3][tid];
            // a wait that ran out leaves NaN, which the answer then shows
            my_stats[tid] = s_failed ? make_float2(NAN, NAN)
                            : l > 0.f || isnan(l) ? make_float2(s_ref[tid], l)
                                                  : make_float2(-INFINITY, 0.f);
        }
        if (!s_failed)
            for (int m = 0; m * 128 < a.D; ++m) {
                const int d = m * 128 + key;
                float* to = part + ((bh * p.splits + split) * a.R + row0) * a.D + d;
                float o[RT], lo[RT];
                tmem_ld<RT>(lanes + (2 + 2 * m) * RT, o);
                tmem_ld<RT>(lanes + (3 + 2 * m) * RT, lo);
                if (d < a.D)
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        if (r < rows) to[(int64_t)r * a.D] = fmaf(lo[r], 1.f / kApart, o[r]);
            }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, kNarrowCols);
    }
}

// The same run for a tile of up to 128 rows, where rows fill the M side: S = Q K^T,
// and a thread holds one row's logits of half a tile of keys, so that maxima and sums need no
// exchange but that of two threads.  The weights go back into tensor memory, over the
// logits they came from (hi and lo parts side by side), and are the A operand of O += P V there:
// with them in shared memory its bandwidth was the limit (288 KB a tile and 128 rows, 2300 of
// 4300 cycles).
template <class T>
__global__ void __launch_bounds__(kWideThreads, 1)
    attend_wide_kernel(AttendArgs a, AttendPlan p, const T* q,
                       const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, float2* stats, float* part) {
    constexpr int RT = 128, kHalf = kTile / 2;
    constexpr float kLift = Pair<T>::kLift, kMost = Pair<T>::kMost, kApart = Pair<T>::kApart;
    extern __shared__ char smem_raw[];
    __shared__ uint64_t bars[2 * kMaxStages + 5];
    __shared__ uint32_t s_tmem;
    __shared__ int s_failed;
    __shared__ float s_pair[2][RT];  // what the two threads of a row tell each other
    const int lane = threadIdx.x & 31, warp = uniform((int)threadIdx.x >> 5);
    const int rt = blockIdx.x % p.row_tiles;
    const int64_t rest = blockIdx.x / p.row_tiles;
    const int split = (int)(rest % p.splits);
    const int64_t bh = rest / p.splits;
    const int b = (int)(bh / a.Hkv), h = (int)(bh % a.Hkv);
    const int64_t row0 = (int64_t)rt * RT;
    const int rows = (int)(a.R - row0 < RT ? a.R - row0 : RT);
    float2* my_stats = stats + (bh * p.splits + split) * a.R + row0;

    pdl_wait();
    const int64_t n = uniform(cache_length(a, b));
    // keys that the tile's last row sees, and this run's tiles among them
    int64_t seen = n - a.Sq + 1 + (row0 + rows - 1) / a.G;
    seen = seen < 0 ? 0 : seen;
    const int64_t all_tiles = (seen + kTile - 1) / kTile;
    const int64_t per = (all_tiles + p.splits - 1) / p.splits;
    const int64_t first = split * per;
    const int tiles = (int)(all_tiles - first < per ? all_tiles - first : per);
    if (tiles <= 0) {
        if (threadIdx.x < rows) my_stats[threadIdx.x] = make_float2(-INFINITY, 0.f);
        return;
    }

    const int subs = (a.D + 63) / 64;
    const uint32_t sub_bytes = kTile * 128, stage_bytes = subs * sub_bytes;
    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t q_at = ring + p.stages * stage_bytes;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kMaxStages,
                   s_done = empty + 8 * kMaxStages, p_full = s_done + 16, p_used = p_full + 16;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        mbar_init(s_done, 1);
        mbar_init(s_done + 8, 1);
        mbar_init(p_full, 256);  // one per half: the softmax may be a tile ahead of the product
        mbar_init(p_full + 8, 256);
        mbar_init(p_used, 1);
        fence_barrier_init();
        s_failed = 0;
    }
    if (warp == 1) tmem_alloc(smem_addr(&s_tmem), 512);
    load_rows<T, RT>(a, q, b, h, row0, rows, q_at, threadIdx.x, kWideThreads);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // logits (then weights) of two tiles, then the outputs; where there is room for two (and for
    // fp16 only), those of the weights' hi and lo parts apart
    const uint32_t tmem = uniform(s_tmem), o_col = tmem + 2 * kTile;
    const bool two = kApart != 1.f && a.D <= 128;
    const uint32_t lo_col = two ? 128 : 0;
    const float apart = two ? kApart : 1.f;
    // the ring's items: K0, K1, V0, K2, V1, ..., V(last)
    const int items = 2 * tiles;
    auto key_item = [](int t) { return t == 0 ? 0 : 2 * t - 1; };
    auto value_item = [&](int t) { return t + 1 < tiles ? 2 * t + 2 : 2 * t + 1; };
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (; issued < items; ++issued) {
                const int s = issued % p.stages, turn = issued / p.stages;
                if (turn > 0) ok = mbar_wait(empty + 8 * s, (turn - 1) & 1);
                if (!ok) break;
                mbar_expect(full + 8 * s, stage_bytes);
                const bool key = issued == 0 || (issued % 2 == 1 && issued < items - 1);
                const int t = key ? (issued + 1) / 2 : (issued - 1) / 2;
                const int y = (int)((first + t) * kTile);
                for (int c = 0; c < subs; ++c)
                    tma_load_4d(ring + s * stage_bytes + c * sub_bytes, key ? &k_map : &v_map,
                                full + 8 * s, c * 64, y, h * (key ? a.kh : a.vh),
                                b * (key ? a.kb : a.vb));
            }
            if (!ok)  // gave up: let the copies in flight land before the block ends
                for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
                    mbar_wait(full + 8 * (i % p.stages), (i / p.stages) & 1);
        }
    } else if (warp == 1) {
        const uint32_t shape_s = mma_shape(Pair<T>::bf16, false, false, RT, kTile);
        const uint32_t shape_o = mma_shape(Pair<T>::bf16, false, true, RT, a.D);
        const uint64_t q_op = operand(q_at, 16, 1024, kSwizzle128);
        auto logits_of = [&](int t) {  // S of tile t into its half
            const int item = key_item(t), s = item % p.stages;
            if (!__all_sync(kAll, mbar_wait(full + 8 * s, (item / p.stages) & 1))) return false;
            tc_fence_after();
            if (elect_one()) {
                key_products<RT>(tmem + (t & 1) * kTile, q_op,
                                 operand(ring + s * stage_bytes, 16, 1024, kSwizzle128), a.D,
                                 shape_s);
                mma_commit(empty + 8 * s);
                mma_commit(s_done + 8 * (t & 1));
            }
            __syncwarp();
            return true;
        };
        ok = logits_of(0) && (tiles == 1 || logits_of(1));
        for (int t = 0; t < tiles && ok; ++t) {
            const int item = value_item(t), s = item % p.stages;
            ok = mbar_wait(full + 8 * s, (item / p.stages) & 1) &&
                 mbar_wait(p_full + 8 * (t & 1), (t >> 1) & 1);
            ok = __all_sync(kAll, ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                // 16 keys at a time: 8 columns of weights; each half of the tile has its hi
                // parts in 32 columns and its lo parts in the next 32
                const uint64_t v = operand(ring + s * stage_bytes, sub_bytes, 1024, kSwizzle128);
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk) {
                    const uint32_t w = tmem + (t & 1) * kTile + (kk >> 2) * kHalf + (kk & 3) * 8;
                    mma_f16_ta(o_col, w, v + advance(kk * 2048), shape_o, t + kk > 0);
                    mma_f16_ta(o_col + lo_col, w + 32, v + advance(kk * 2048), shape_o, !two || t + kk > 0);
                }
                mma_commit(empty + 8 * s);
                mma_commit(p_used);
            }
            __syncwarp();
            // the next logits of this half go over weights that the product has read
            if (t + 2 < tiles) ok = __all_sync(kAll, mbar_wait(p_used, t & 1)) && logits_of(t + 2);
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) / 4;
        const int row = quarter * 32 + lane;  // of the tile
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const bool busy = quarter * 32 < rows;  // warps without a row only keep step
        // keys that the row sees, and the fewest that any row does, from the run's first
        const int64_t most = (int64_t)tiles * kTile;
        int64_t lim64 = n - a.Sq + 1 + (row0 + row) / a.G - first * kTile;
        const int lim = (int)(row >= rows || lim64 > most ? most : lim64 < 0 ? 0 : lim64);
        lim64 = n - a.Sq + 1 + row0 / a.G - first * kTile;
        const int least = (int)(lim64 > most ? most : lim64 < 0 ? 0 : lim64);
        float ref = 0.f, sum = 0.f;
        bool fresh = true;  // the row has seen no key yet
        for (int t = 0; t < tiles; ++t) {
            ok = ok && mbar_wait(s_done + 8 * (t & 1), (t >> 1) & 1);
            ok = __all_sync(kAll, ok);
            tc_fence_after();
            const uint32_t at = lanes + (t & 1) * kTile + half * kHalf;
            const int key0 = t * kTile + half * kHalf;
            const int64_t j0 = (first + t) * kTile;
            if (j0 + kTile > n && half == 0) {
                // value rows behind the cache's end may hold anything: 0 x NaN is NaN
                const int item = value_item(t), s = item % p.stages;
                ok = ok && mbar_wait(full + 8 * s, (item / p.stages) & 1);
                if (ok && j0 + row >= n)
                    for (int c = 0; c < subs * 8; ++c)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         ring + s * stage_bytes + (c >> 3) * sub_bytes + row * 128 +
                                         (c & 7) * 16),
                                     "r"(0)
                                     : "memory");
                fence_async_smem();
                __syncwarp();
            }
            if (busy) {
                float x[kHalf];
#pragma unroll
                for (int c = 0; c < kHalf; c += 32)
                    tmem_ld<32>(at + c, *reinterpret_cast<float(*)[32]>(x + c));
#pragma unroll
                for (int c = 0; c < kHalf; ++c) x[c] = fmaf(x[c], a.scale_log2, -ref);
                if (key0 + kHalf > least)
#pragma unroll
                    for (int c = 0; c < kHalf; ++c)
                        if (key0 + c >= lim) x[c] = -INFINITY;
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kHalf; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
                const float by = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                // one answer for the two warps that share these rows
                uint32_t raise;
                asm volatile(
                    "{\n\t.reg .pred u, v;\n\tsetp.ne.u32 u, %1, 0;\n\t"
                    "barrier.cta.red.or.pred v, %2, 64, u;\n\tselp.u32 %0, 1, 0, v;\n\t}"
                    : "=r"(raise)
                    : "r"(by > (fresh ? -INFINITY : kMost) ? 1u : 0u), "r"(2 + quarter)
                    : "memory");
                if (raise) {
                    s_pair[half][row] = by;
                    if (t > 0) {  // the outputs so far are complete
                        ok = ok && mbar_wait(p_used, (t - 1) & 1);
                        ok = __all_sync(kAll, ok);
                        tc_fence_after();
                    }
                    asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter) : "memory");
                    const float both = fmaxf(s_pair[0][row], s_pair[1][row]);
                    asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter) : "memory");
                    const bool none = fresh && both == -INFINITY;
                    const float up = none ? 0.f : fresh ? both - kLift : fmaxf(both - kLift, 0.f);
                    const float scale = fresh ? 0.f : ex2_ftz(-up);
                    ref += up;
                    fresh = none;
                    sum *= scale;
#pragma unroll
                    for (int c = 0; c < kHalf; ++c) x[c] -= up;
                    if (t > 0)  // each thread rescales half of the row's outputs
                        for (uint32_t col = 0; col <= lo_col; col += 128)
                            for (int c = half * 16; c < a.D; c += 32) {
                                float o[16];
                                tmem_ld<16>(lanes + 2 * kTile + col + c, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= scale;
                                tmem_st<16>(lanes + 2 * kTile + col + c, o);
                            }
                }
                float part_sum[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t hi[kHalf / 2], lo[kHalf / 2];
#pragma unroll
                for (int c = 0; c < kHalf; c += 2) {
                    const float u = ex2_ftz(x[c]), w = ex2_ftz(x[c + 1]);
                    part_sum[c & 3] += u;
                    part_sum[(c & 3) + 1] += w;
                    Pair<T>::split(u, w, apart, &hi[c / 2], &lo[c / 2]);
                }
                sum += (part_sum[0] + part_sum[1]) + (part_sum[2] + part_sum[3]);
                tmem_st<32>(at, hi);
                tmem_st<32>(at + 32, lo);
            }
            tc_fence_before();
            mbar_arrive(p_full + 8 * (t & 1));
        }
        // both products that may be under way: of a barrier two phases behind, the last one
        // would look complete
        if (ok && tiles > 1) ok = mbar_wait(p_used, (tiles - 2) & 1);
        if (ok) ok = mbar_wait(p_used, (tiles - 1) & 1);
        if (!ok) s_failed = 1;
        s_pair[half][row] = sum;
        softmax_sync<256>();
        tc_fence_after();
        if (half == 0 && row < rows) {
            const float l = s_pair[0][row] + s_pair[1][row];
            // a wait that ran out leaves NaN, which the answer then shows
            my_stats[row] = s_failed ? make_float2(NAN, NAN)
                            : l > 0.f || isnan(l) ? make_float2(ref, l)
                                                  : make_float2(-INFINITY, 0.f);
        }
        if (!s_failed && busy) {
            float* to = part + ((bh * p.splits + split) * a.R + row0 + row) * a.D;
            for (int c = half * 16; c < a.D; c += 32) {
                float o[16];
                tmem_ld<16>(lanes + 2 * kTile + c, o);
                if (two) {
                    float lo[16];
                    tmem_ld<16>(lanes + 2 * kTile + lo_col + c, lo);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = fmaf(lo[i], 1.f / kApart, o[i]);
                }
                if (row < rows)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4*>(to + c + i) =
                            make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

// log2 of the sum of 2^x over all of a row's runs, by one warp; +inf for a row that saw
// nothing.
__device__ __forceinline__ float row_lse(const float2* stats, int splits, int64_t R, int lane) {
    float m = -INFINITY, l = 0.f;
    bool bad = false;
    for (int s = lane; s < splits; s += 32) {
        const float2 x = stats[s * R];
        bad |= isnan(x.x) || isnan(x.y);
        if (!(x.y > 0.f)) continue;
        const float to = fmaxf(m, x.x);
        l = l * ex2_ftz(m - to) + x.y * ex2_ftz(x.x - to);
        m = to;
    }
    if (__any_sync(kAll, bad)) return NAN;
    float all = m;
#pragma unroll
    for (int d = 16; d; d >>= 1) all = fmaxf(all, __shfl_xor_sync(kAll, all, d));
    l = m > -INFINITY ? l * ex2_ftz(m - all) : 0.f;
#pragma unroll
    for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(kAll, l, d);
    return l > 0.f ? all + log2f(l) : INFINITY;
}

// Scores of the kJoinKeys keys from j0 on out of kept logits, W float4 of rows a key (a
// row that does not see a key has left -inf).  The logits are fetched before the rows'
// logs are known.
template <int W>
__device__ __forceinline__ void kept_scores(const AttendArgs& a, const AttendPlan& p, int64_t bh,
                                            int64_t b, int64_t h, int64_t j0, int64_t n,
                                            const float2* stats, const float* logits,
                                            const float* score_in, float* score_out, float* lse) {
    constexpr int kOwn = kJoinKeys / kJoinThreads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float4 x[kOwn][W];
    float old[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int64_t j = j0 + i * kJoinThreads + threadIdx.x;
        old[i] = 0.f;
        if (j >= n) continue;
        const float4* at = reinterpret_cast<const float4*>(logits + (bh * a.N + j) * (4 * W));
#pragma unroll
        for (int w = 0; w < W; ++w) x[i][w] = at[w];
        if (score_in != nullptr) old[i] = score_in[b * a.sib + h * a.sih + j];
    }
    for (int r = warp; r < 4 * W; r += kJoinThreads / 32) {
        const float v = r < a.R ? row_lse(stats + bh * p.splits * a.R + r, p.splits, a.R, lane)
                                : INFINITY;
        if (lane == 0) lse[r] = v;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int64_t j = j0 + i * kJoinThreads + threadIdx.x;
        if (j >= n) continue;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float4 m = *reinterpret_cast<const float4*>(lse + 4 * w);
            s += ex2_ftz(x[i][w].x - m.x) + ex2_ftz(x[i][w].y - m.y);
            s += ex2_ftz(x[i][w].z - m.z) + ex2_ftz(x[i][w].w - m.w);
        }
        score_out[b * a.sob + h * a.soh + j] = old[i] + s;
    }
}

// Joins the runs.  The first blocks turn kept logits into scores; the others join the
// outputs, one warp a row, and leave each row's log of the sum.
template <class T>
__global__ void __launch_bounds__(kJoinThreads)
    attend_join_kernel(AttendArgs a, AttendPlan p, int64_t score_blocks, int key_blocks,
                       const float2* stats, const float* part, const float* logits,
                       const float* score_in, float* score_out, float* row_logs, T* out) {
    pdl_wait();
    __shared__ alignas(16) float lse[kKeepRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x < score_blocks) {
        const int64_t bh = blockIdx.x / key_blocks, b = bh / a.Hkv, h = bh - b * a.Hkv;
        const int64_t n = cache_length(a, b), j0 = (int64_t)(blockIdx.x % key_blocks) * kJoinKeys;
        if (j0 >= n) return;
        switch (p.RP / 4) {
            case 1: kept_scores<1>(a, p, bh, b, h, j0, n, stats, logits, score_in, score_out, lse); break;
            case 2: kept_scores<2>(a, p, bh, b, h, j0, n, stats, logits, score_in, score_out, lse); break;
            case 3: kept_scores<3>(a, p, bh, b, h, j0, n, stats, logits, score_in, score_out, lse); break;
            default: kept_scores<4>(a, p, bh, b, h, j0, n, stats, logits, score_in, score_out, lse);
        }
        return;
    }
    const int64_t row = (blockIdx.x - score_blocks) * (kJoinThreads / 32) + warp;
    if (row >= (int64_t)a.B * a.Hkv * a.R) return;
    const int64_t bh = row / a.R, r = row - bh * a.R, b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int64_t tok = r / a.G, g = r - tok * a.G;
    const float2* st = stats + bh * p.splits * a.R + r;
    const float top = row_lse(st, p.splits, a.R, lane);
    if (lane == 0 && !p.keep) row_logs[row] = top;
    T* to = out + ((b * a.Sq + tok) * a.Hkv * a.G + h * a.G + g) * a.D;
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int d0 = 0; d0 < a.D; d0 += 128) {
        const int d = d0 + lane * 4;
        float4 acc = none;
        for (int s0 = 0; s0 < p.splits; s0 += 32) {
            const float2 x = s0 + lane < p.splits ? st[(s0 + lane) * a.R] : make_float2(0.f, 0.f);
            // a run in which the row saw nothing has written no outputs: weight 0, not read
            const float w = x.y > 0.f ? ex2_ftz(x.x - top) : 0.f;
            const int cnt = p.splits - s0 < 32 ? p.splits - s0 : 32;
#pragma unroll 8
            for (int s = 0; s < cnt; ++s) {
                const float ws = __shfl_sync(kAll, w, s);
                const float4 o = ws > 0.f && d < a.D
                                     ? *reinterpret_cast<const float4*>(
                                           part + ((bh * p.splits + s0 + s) * a.R + r) * a.D + d)
                                     : none;
                acc.x = fmaf(ws, o.x, acc.x);
                acc.y = fmaf(ws, o.y, acc.y);
                acc.z = fmaf(ws, o.z, acc.z);
                acc.w = fmaf(ws, o.w, acc.w);
            }
        }
        if (isnan(top)) acc = make_float4(NAN, NAN, NAN, NAN);
        if (d < a.D) {
            Pack<T, 4> o;
            o.v[0] = narrow<T>(acc.x);
            o.v[1] = narrow<T>(acc.y);
            o.v[2] = narrow<T>(acc.z);
            o.v[3] = narrow<T>(acc.w);
            *reinterpret_cast<Pack<T, 4>*>(to + d) = o;
        }
    }
}

// Scores where the logits were not kept.  A block streams a run of key tiles past
// up to kScoreRows rows that stay in shared memory (more rows: once per such group); the
// two halves of the softmax warps take the tiles in turn, each with its own half of tensor
// memory, and a thread sums one key's weights over the rows, whose logs it knows.
template <class T>
__global__ void __launch_bounds__(kScoreThreads, 2)
    attend_score_kernel(AttendArgs a, ScorePlan p, const T* q,
                        const __grid_constant__ CUtensorMap k_map, const float* row_logs,
                        const float* score_in, float* score_out) {
    extern __shared__ char smem_raw[];
    __shared__ uint64_t bars[2 * kMaxStages + 5];
    __shared__ uint32_t s_tmem;
    __shared__ alignas(16) float s_log[kScoreRows];
    const int lane = threadIdx.x & 31, warp = uniform((int)threadIdx.x >> 5);
    const int64_t bh = blockIdx.x / p.blocks;
    const int b = (int)(bh / a.Hkv), h = (int)(bh % a.Hkv);
    pdl_wait();
    const int64_t n = uniform(cache_length(a, b));
    // the sequence's tiles shared out evenly among its blocks
    const int64_t all = (n + kTile - 1) / kTile, per = (all + p.blocks - 1) / p.blocks;
    const int64_t first = blockIdx.x % p.blocks * per;
    const int tiles = (int)(all - first < per ? all - first : per);
    if (tiles <= 0) return;
    const int subs = (a.D + 63) / 64;
    const uint32_t sub_bytes = kTile * 128, tile_bytes = subs * sub_bytes;
    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u, q_at = ring + p.stages * tile_bytes;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kMaxStages,
                   q_full = empty + 8 * kMaxStages, done = q_full + 8, used = done + 16;
    // groups of rows that see some key here: the first key sees the most rows
    const int64_t past = first * kTile - (n - a.Sq);
    const int64_t rg0 = (past > 0 ? past * a.G : 0) / kScoreRows,
                  rgs = (a.R + kScoreRows - 1) / kScoreRows;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        mbar_init(q_full, 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(done + 8 * i, 1);
            mbar_init(used + 8 * i, 128);
        }
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(smem_addr(&s_tmem), 2 * kScoreRows);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(s_tmem);
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int64_t rg = rg0; rg < rgs && ok; ++rg)
                for (int t = 0; t < tiles; ++t, ++issued) {
                    const int s = issued % p.stages, turn = issued / p.stages;
                    if (turn > 0) ok = mbar_wait(empty + 8 * s, (turn - 1) & 1);
                    if (!ok) break;
                    mbar_expect(full + 8 * s, tile_bytes);
                    for (int c = 0; c < subs; ++c)
                        tma_load_4d(ring + s * tile_bytes + c * sub_bytes, &k_map, full + 8 * s, c * 64,
                                    (int)((first + t) * kTile), h * a.kh, b * a.kb);
                }
            if (!ok)  // gave up: let the copies in flight land before the block ends
                for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
                    mbar_wait(full + 8 * (i % p.stages), (i / p.stages) & 1);
        }
    } else if (warp == 1) {
        const uint64_t q_op = operand(q_at, 16, 1024, kSwizzle128);
        int item = 0, turns[2] = {0, 0};
        for (int64_t rg = rg0; rg < rgs && ok; ++rg) {
            const int rows = (int)(a.R - rg * kScoreRows < kScoreRows ? a.R - rg * kScoreRows : kScoreRows);
            const uint32_t shape = mma_shape(Pair<T>::bf16, false, false, kTile, (rows + 31) & ~31);
            ok = __all_sync(kAll, mbar_wait(q_full, (rg - rg0) & 1));
            for (int t = 0; t < tiles && ok; ++t, ++item) {
                const int s = item % p.stages, half = t & 1;
                ok = mbar_wait(full + 8 * s, (item / p.stages) & 1);
                if (ok && turns[half] > 0) ok = mbar_wait(used + 8 * half, (turns[half] - 1) & 1);
                ok = __all_sync(kAll, ok);
                if (!ok) break;
                ++turns[half];
                tc_fence_after();
                if (elect_one()) {
                    key_products<kScoreRows>(tmem + half * kScoreRows,
                                             operand(ring + s * tile_bytes, 16, 1024, kSwizzle128),
                                             q_op, a.D, shape);
                    mma_commit(empty + 8 * s);
                    mma_commit(done + 8 * half);
                }
                __syncwarp();
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) / 4, key = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + half * kScoreRows;
        const float* in = score_in != nullptr ? score_in + b * a.sib + h * a.sih : nullptr;
        float* out = score_out + b * a.sob + h * a.soh;
        int turn = 0;
        for (int64_t rg = rg0; rg < rgs; ++rg) {
            const int64_t row0 = rg * kScoreRows;
            const int rows = (int)(a.R - row0 < kScoreRows ? a.R - row0 : kScoreRows);
            // both halves are done with the rows before, and with them the products
            softmax_sync<256>();
            load_rows<T, kScoreRows>(a, q, b, h, row0, rows, q_at, threadIdx.x - 64, 256);
            for (int r = threadIdx.x - 64; r < kScoreRows; r += 256)
                s_log[r] = r < rows ? row_logs[bh * a.R + row0 + r] : INFINITY;
            fence_async_smem();
            softmax_sync<256>();
            mbar_arrive(q_full);
            for (int t = half; t < tiles; t += 2) {
                const int64_t j = (first + t) * kTile + key;
                // rows from this one on (of the group) see the key
                const int64_t past_j = j - (n - a.Sq);
                const int64_t from64 = (past_j > 0 ? past_j * a.G : 0) - row0;
                const int from = from64 <= 0 ? 0 : from64 < kScoreRows ? (int)from64 : kScoreRows;
                float old = 0.f;
                if (j < n) old = rg > rg0 ? out[j] : in != nullptr ? in[j] : 0.f;
                if (ok) ok = mbar_wait(done + 8 * half, turn & 1);
                ++turn;
                ok = __all_sync(kAll, ok);
                float s = 0.f;
                if (ok) {
                    tc_fence_after();
                    for (int c = 0; c < rows; c += 32) {
                        float x[32];
                        tmem_ld<32>(lanes + c, x);
                        // rows that do not see the key, and those of zeros past the last one (whose
                        // product with an infinite key is NaN), count nothing
                        if (__any_sync(kAll, from > c) || c + 32 > rows) {
#pragma unroll
                            for (int r = 0; r < 32; ++r)
                                s += c + r >= from && c + r < rows
                                         ? ex2_ftz(fmaf(x[r], a.scale_log2, -s_log[c + r]))
                                         : 0.f;
                        } else {
#pragma unroll
                            for (int r = 0; r < 32; ++r)
                                s += ex2_ftz(fmaf(x[r], a.scale_log2, -s_log[c + r]));
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(used + 8 * half);
                }
                if (j < n) out[j] = ok ? old + s : NAN;  // a wait that ran out leaves NaN
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, 2 * kScoreRows);
    }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

bool attend_sizes_ok(int64_t B, int64_t Sq, int64_t Hq, int64_t Hkv, int64_t N, int64_t D) {
    const int64_t big = int64_t(1) << 31;
    return B >= 1 && Sq >= 1 && Hq >= 1 && Hkv >= 1 && N >= 1 && B < 65536 && Sq < 65536 &&
           Hq < 65536 && Hkv <= Hq && N < big - kTile && Hq % Hkv == 0 && D >= 16 && D <= 256 &&
           D % 16 == 0 && B * Sq < big / Hq && B * Hkv * ((N + 127) / 128) < big / 16;
}

AttendPlan make_plan(int64_t B, int64_t Sq, int64_t Hq, int64_t Hkv, int64_t N, int64_t D) {
    AttendPlan p{};
    const int64_t R = Sq * (Hq / Hkv), bh = B * Hkv;
    p.keep = R <= kKeepRows;
    p.rt = p.keep ? kKeepRows : 128;
    p.row_tiles = (int)((R + p.rt - 1) / p.rt);
    const int subs = (int)(D + 63) / 64, stage = subs * kTile * 128;
    // few rows: the weights too, and since V^T is read 128 rows at a time, past an odd last
    // block of 64 columns its (unused) rows are whatever follows, which has to be there
    const int fixed = 1024 + subs * p.rt * 128 +
                      (p.keep ? p.rt * 512 + (subs % 2 ? kTile * 128 : 0) : 0);
    // few rows: two blocks an SM where three stages fit half of it
    const bool two = p.keep && fixed + 3 * stage <= 112 * 1024;
    const int room = (two ? 112 : kBlockSmem) * 1024 - fixed;
    p.stages = room / stage < kMaxStages ? room / stage : kMaxStages;
    p.smem = fixed + p.stages * stage;
    // Runs.  x blocks a run over `slots` places: with equal lengths they take whole waves of
    // L tiles and a block's own time, with lengths between a fifth and all of N about 0.6 of
    // that and one run more at the end; joining takes about 0.03 tiles a run.  The lengths are
    // the device's to know, so the cheapest sum of both (the first counted twice) is taken.
    // Against the best of 22 forced numbers of runs, for 25 batches (1 to 32 sequences of 1024 to
    // 131072 keys, 1 to 64 tokens, equal and ragged): within 3% for 16 of them, 10% for 23, and
    // 19% for one sequence of 4099 (33 runs for 18: 14.4 us for 12.1) and of 131072 keys (171
    // for 128: 31.3 for 26.3), where joining costs more than assumed.
    const int64_t tiles = (N + kTile - 1) / kTile, slots = kSms * (two ? 2 : 1), x = bh * p.row_tiles;
    const double own = p.keep ? 1.5 : 4.0;  // a block's start and end, in tiles
    int64_t splits = 1;
    double least = 1e300;
    for (int64_t t = 1; t <= tiles && t <= kMostRuns; ++t) {
        const double run = (double)((tiles + t - 1) / t), waves = (double)((x * t + slots - 1) / slots),
                     even = waves * (run + own),
                     uneven = (double)(x * t) / (double)slots * (0.6 * run + own) + run;
        const double cost = 2.0 * even + uneven + 0.09 * (double)t;
        if (cost < least) {
            least = cost;
            splits = t;
        }
    }
    p.splits = (int)splits;
    p.RP = (R + 3) / 4 * 4;
    p.off_lse = up256((size_t)(bh * p.splits * R) * 8);
    p.off_part = p.off_lse + up256((size_t)(bh * R) * 4);
    p.off_logits = p.off_part + up256((size_t)(bh * p.splits * R) * (size_t)D * 4);
    p.bytes = p.off_logits + (p.keep ? up256((size_t)(bh * N) * (size_t)p.RP * 4) : 0);
    return p;
}

ScorePlan make_score_plan(int64_t bh, int64_t N, int64_t D) {
    ScorePlan p{};
    const int subs = (int)(D + 63) / 64, tile = subs * kTile * 128, fixed = 1024 + subs * kScoreRows * 128;
    // two blocks an SM where two stages fit half of it
    const bool two = fixed + 2 * tile <= 112 * 1024;
    const int room = (two ? 112 : kBlockSmem) * 1024 - fixed;
    p.stages = room / tile < kMaxStages ? room / tile : kMaxStages;
    p.smem = fixed + p.stages * tile;
    const int64_t tiles = (N + kTile - 1) / kTile, slots = kSms * (two ? 2 : 1);
    // one wave of blocks, or blocks of at most 16 tiles where there are more heads
    int64_t blocks = slots / bh;
    if (blocks < (tiles + 15) / 16 && bh * ((tiles + 15) / 16) > 2 * slots) blocks = (tiles + 15) / 16;
    p.blocks = (int)(blocks < 1 ? 1 : blocks < tiles ? blocks : tiles);
    return p;
}

// The driver's tensor-map encoder, looked up once.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
    static std::atomic<void*> fn{nullptr};
    void* f = fn.load(std::memory_order_acquire);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return (EncodeFn)f;
}

// A cache as (B, Hkv, N, D), boxes of 128 rows by 64 elements, swizzled by 128 bytes.  A
// dimension that repeats one and the same memory (stride 0) is mapped with length 1.
bool cache_map(CUtensorMap* map, int dtype, const void* base, int64_t B, int64_t H, int64_t N,
               int64_t D, int64_t sb, int64_t sh, int64_t sr, int* use_h, int* use_b) {
    const EncodeFn encode = encoder();
    if (encode == nullptr) return false;
    *use_h = sh > 0 && H > 1;
    *use_b = sb > 0 && B > 1;
    const int64_t rows = sr > 0 ? N : 1;
    if (rows < N) return false;  // every row the same memory: not a cache
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)(*use_h ? H : 1),
                                (cuuint64_t)(*use_b ? B : 1)};
    const cuuint64_t strides[3] = {(cuuint64_t)sr * 2, (cuuint64_t)(*use_h ? sh : sr) * 2,
                                   (cuuint64_t)(*use_b ? sb : sr) * 2};
    const cuuint32_t box[4] = {64, kTile, 1, 1}, step[4] = {1, 1, 1, 1};
    return encode(map, dtype == LAPSUM_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  4, const_cast<void*>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T>
cudaError_t launch_attend(const AttendArgs& a, const AttendPlan& p, const void* q,
                          const CUtensorMap& k, const CUtensorMap& v, char* ws,
                          const float* score_in, float* score_out, void* out, cudaStream_t st) {
    float2* stats = (float2*)ws;
    float* row_logs = (float*)(ws + p.off_lse);
    float* part = (float*)(ws + p.off_part);
    float* logits = (float*)(ws + p.off_logits);
    cudaError_t e;
    {
        ProfScope prof("attend_split", st);
        static std::atomic<unsigned long long> done{0};
        once_per_device(done, [] {
            cudaFuncSetAttribute(attend_narrow_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kBlockSmem * 1024);
            cudaFuncSetAttribute(attend_wide_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kBlockSmem * 1024);
            cudaFuncSetAttribute(attend_score_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kBlockSmem * 1024);
        });
        const dim3 blocks((unsigned)((int64_t)a.B * a.Hkv * p.splits * p.row_tiles));
        e = p.keep ? launch_pdl(attend_narrow_kernel<T>, blocks, dim3(kNarrowThreads), (size_t)p.smem, st,
                                a, p, (const T*)q, k, v, stats, part, logits)
                   : launch_pdl(attend_wide_kernel<T>, blocks, dim3(kWideThreads), (size_t)p.smem, st, a,
                                p, (const T*)q, k, v, stats, part);
    }
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)a.B * a.Hkv * a.R;
    {
        ProfScope prof("attend_join", st);
        const int key_blocks = (int)((a.N + kJoinKeys - 1) / kJoinKeys);
        const int64_t score_blocks = p.keep ? (int64_t)a.B * a.Hkv * key_blocks : 0;
        e = launch_pdl(attend_join_kernel<T>, dim3((unsigned)(score_blocks + (rows + 7) / 8)),
                       dim3(kJoinThreads), 0, st, a, p, score_blocks, key_blocks,
                       (const float2*)stats, (const float*)part, (const float*)logits, score_in,
                       score_out, row_logs, (T*)out);
    }
    if (e != cudaSuccess || p.keep) return e;
    ProfScope prof("attend_score", st);
    const ScorePlan sp = make_score_plan((int64_t)a.B * a.Hkv, a.N, a.D);
    return launch_pdl(attend_score_kernel<T>, dim3((unsigned)((int64_t)a.B * a.Hkv * sp.blocks)),
                      dim3(kScoreThreads), (size_t)sp.smem, st, a, sp, (const T*)q, k,
                      (const float*)row_logs, score_in, score_out);
}

}  // namespace
}  // namespace lapsum

using namespace lapsum;

extern "C" size_t lapsum_attend_workspace_bytes(int64_t B, int64_t Sq, int64_t Hq, int64_t Hkv,
                                                int64_t N, int64_t D) {
    if (!attend_sizes_ok(B, Sq, Hq, Hkv, N, D)) return 0;
    return make_plan(B, Sq, Hq, Hkv, N, D).bytes;
}

extern "C" int lapsum_attend_accumulate(const void* q, const void* k, const void* v, int dtype,
                                        const int32_t* lengths, const int64_t* strides, int64_t B,
                                        int64_t Sq, int64_t Hq, int64_t Hkv, int64_t N, int64_t D,
                                        float scale, const float* score_in, float* score_out,
                                        void* out, void* ws, size_t ws_bytes, void* stream) {
    if (q == nullptr || k == nullptr || v == nullptr || lengths == nullptr || strides == nullptr ||
        score_out == nullptr || out == nullptr)
        return LAPSUM_EINVAL;
    if (dtype != LAPSUM_DTYPE_BF16 && dtype != LAPSUM_DTYPE_F16) return LAPSUM_EINVAL;
    if (!attend_sizes_ok(B, Sq, Hq, Hkv, N, D) || !std::isfinite(scale)) return LAPSUM_EINVAL;
    // the stride of a dimension of one element means nothing
    const int64_t size[13] = {B, Hq, Sq, B, Hkv, N, B, Hkv, N, B, Hkv, B, Hkv};
    int64_t own[13];
    for (int i = 0; i < 13; ++i) {
        own[i] = size[i] > 1 ? strides[i] : 0;
        if (own[i] < 0 || (i < 9 && own[i] % 8 != 0)) return LAPSUM_EINVAL;
    }
    strides = own;
    // rows of one cache may repeat over heads and sequences, but not over its keys
    if (N > 1 && (strides[5] < D || strides[8] < D)) return LAPSUM_EINVAL;
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(out, 16) ||
        !aligned_to(lengths, 4) || !aligned_to(score_in, 4) || !aligned_to(score_out, 4))
        return LAPSUM_EINVAL;
    const AttendPlan p = make_plan(B, Sq, Hq, Hkv, N, D);
    if (ws == nullptr || !aligned_to(ws, 256) || ws_bytes < p.bytes) return LAPSUM_EWORKSPACE;
    AttendArgs a{};
    a.qb = strides[0];
    a.qh = strides[1];
    a.qr = strides[2];
    a.sib = strides[9];
    a.sih = strides[10];
    a.sob = strides[11];
    a.soh = strides[12];
    a.N = N;
    a.B = (int)B;
    a.Sq = (int)Sq;
    a.Hkv = (int)Hkv;
    a.D = (int)D;
    a.G = (int)(Hq / Hkv);
    a.R = Sq * a.G;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    a.lengths = lengths;
    CUtensorMap k_map, v_map;
    const int64_t row = D < 8 ? 8 : D;  // a row stride for caches of one row
    if (!cache_map(&k_map, dtype, k, B, Hkv, N, D, strides[3], strides[4],
                   N > 1 ? strides[5] : row, &a.kh, &a.kb) ||
        !cache_map(&v_map, dtype, v, B, Hkv, N, D, strides[6], strides[7],
                   N > 1 ? strides[8] : row, &a.vh, &a.vb))
        return LAPSUM_ECUDA;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e =
        dtype == LAPSUM_DTYPE_BF16
            ? launch_attend<__nv_bfloat16>(a, p, q, k_map, v_map, (char*)ws, score_in, score_out,
                                           out, st)
            : launch_attend<__half>(a, p, q, k_map, v_map, (char*)ws, score_in, score_out, out, st);
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}
