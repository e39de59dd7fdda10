// Attention over a cache that also accumulates, per key, the weight that the
// queries gave it.  Entry point: lapsum_attend_accumulate (include/lapsum.h).
//
// For each sequence b, key/value head h and query row r (a token and one of the
// G = Hq / Hkv query heads that share h):
//     x_j = scale q_r . k_j  over the keys the query sees,  p = softmax(x),
//     out_r = sum_j p_j v_j,   score[b, h, j] += sum_r p_{r, j}.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "elements.cuh"
#include "lapsum_common.cuh"
#include "lapsum_kernels.h"

namespace lapsum {
namespace {

constexpr int kAttThreads = 128;
constexpr unsigned kAll = 0xffffffffu;

struct AttendArgs {
    int64_t qb, qh, qr, kb, kh, kr, vb, vh, vr, sib, sih, sob, soh;
    int64_t B, Sq, Hq, Hkv, N;
    int D, G;
    float scale;
    const int32_t* lengths;
};

__device__ __forceinline__ int64_t cache_length(const AttendArgs& a, int64_t b) {
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n > a.N ? a.N : n;
}

// One block per query row: logits into the workspace, then the weighted sum.
template <class T>
__global__ void __launch_bounds__(kAttThreads)
    attend_rows_kernel(AttendArgs a, const T* q, const T* k, const T* v, T* out, float* logits,
                       float* lse) {
    pdl_wait();
    __shared__ float sq[256], red[kAttThreads / 32];
    const int64_t row = blockIdx.x;  // ((b * Sq) + i) * Hq + head
    const int64_t head = row % a.Hq, i = row / a.Hq % a.Sq, b = row / a.Hq / a.Sq, h = head / a.G;
    const int64_t n = cache_length(a, b);
    const int64_t see = n - a.Sq + i + 1 < 0 ? 0 : n - a.Sq + i + 1;
    for (int d = threadIdx.x; d < a.D; d += kAttThreads)
        sq[d] = widen(q[b * a.qb + i * a.qr + head * a.qh + d]) * a.scale;
    __syncthreads();
    float* x = logits + row * a.N;
    const T* kp = k + b * a.kb + h * a.kh;
    const T* vp = v + b * a.vb + h * a.vh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float m = -INFINITY;
    for (int64_t j = threadIdx.x; j < see; j += kAttThreads) {
        float s = 0.f;
        for (int d = 0; d < a.D; ++d) s = fmaf(sq[d], widen(kp[j * a.kr + d]), s);
        x[j] = s;
        m = fmaxf(m, s);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, d));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
    float l = 0.f;
    for (int64_t j = threadIdx.x; j < see; j += kAttThreads) l += expf(x[j] - m);
#pragma unroll
    for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(kAll, l, d);
    if (lane == 0) red[warp] = l;
    __syncthreads();
    l = red[0] + red[1] + red[2] + red[3];
    if (threadIdx.x == 0) lse[row] = see > 0 ? m + logf(l) : INFINITY;
    for (int d = threadIdx.x; d < a.D; d += kAttThreads) {
        float o = 0.f;
        for (int64_t j = 0; j < see; ++j) o = fmaf(expf(x[j] - m), widen(vp[j * a.vr + d]), o);
        out[row * a.D + d] = narrow<T>(see > 0 ? o / l : 0.f);
    }
}

__global__ void __launch_bounds__(kAttThreads)
    attend_score_kernel(AttendArgs a, const float* logits, const float* lse, const float* score_in,
                        float* score_out) {
    pdl_wait();
    const int64_t bh = blockIdx.y + (int64_t)gridDim.y * blockIdx.z, b = bh / a.Hkv, h = bh % a.Hkv;
    if (b >= a.B) return;
    const int64_t n = cache_length(a, b);
    for (int64_t j = (int64_t)blockIdx.x * kAttThreads + threadIdx.x; j < n;
         j += (int64_t)gridDim.x * kAttThreads) {
        float s = 0.f;
        for (int64_t i = 0; i < a.Sq; ++i) {
            if (j >= n - a.Sq + i + 1) continue;
            for (int g = 0; g < a.G; ++g) {
                const int64_t row = (b * a.Sq + i) * a.Hq + h * a.G + g;
                s += expf(logits[row * a.N + j] - lse[row]);
            }
        }
        const float old = score_in != nullptr ? score_in[b * a.sib + h * a.sih + j] : 0.f;
        score_out[b * a.sob + h * a.soh + j] = old + s;
    }
}

bool attend_sizes_ok(int64_t B, int64_t Sq, int64_t Hq, int64_t Hkv, int64_t N, int64_t D) {
    const int64_t big = int64_t(1) << 31;
    return B >= 1 && Sq >= 1 && Hq >= 1 && Hkv >= 1 && N >= 1 && B < 65536 && Sq < 65536 &&
           Hq < 65536 && N < big && Hq % Hkv == 0 && D >= 16 && D <= 256 && D % 16 == 0 &&
           B * Sq < big / Hq;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace
}  // namespace lapsum

using namespace lapsum;

extern "C" size_t lapsum_attend_workspace_bytes(int64_t B, int64_t Sq, int64_t Hq, int64_t Hkv,
                                                int64_t N, int64_t D) {
    if (!attend_sizes_ok(B, Sq, Hq, Hkv, N, D)) return 0;
    return up256((size_t)(B * Sq * Hq) * 4) + up256((size_t)(B * Sq * Hq) * (size_t)N * 4);
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
    for (int i = 0; i < 13; ++i)
        if (strides[i] < 0 || (i < 9 && strides[i] % 8 != 0)) return LAPSUM_EINVAL;
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(out, 16) ||
        !aligned_to(lengths, 4) || !aligned_to(score_in, 4) || !aligned_to(score_out, 4))
        return LAPSUM_EINVAL;
    if (ws == nullptr || !aligned_to(ws, 256) ||
        ws_bytes < lapsum_attend_workspace_bytes(B, Sq, Hq, Hkv, N, D))
        return LAPSUM_EWORKSPACE;
    AttendArgs a;
    int64_t* s = &a.qb;
    for (int i = 0; i < 13; ++i) s[i] = strides[i];
    a.B = B;
    a.Sq = Sq;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.N = N;
    a.D = (int)D;
    a.G = (int)(Hq / Hkv);
    a.scale = scale;
    a.lengths = lengths;
    cudaStream_t st = (cudaStream_t)stream;
    float* lse = (float*)ws;
    float* logits = (float*)((char*)ws + up256((size_t)(B * Sq * Hq) * 4));
    cudaError_t e;
    {
        ProfScope prof("attend_rows", st);
        e = with_dtype(dtype, [&](auto* tag) {
            using T = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
            return launch_pdl(attend_rows_kernel<T>, dim3((unsigned)(B * Sq * Hq)),
                              dim3(kAttThreads), 0, st, a, (const T*)q, (const T*)k, (const T*)v,
                              (T*)out, logits, lse);
        });
    }
    if (e != cudaSuccess) return LAPSUM_ECUDA;
    ProfScope prof("attend_score", st);
    const int64_t blocks = (N + kAttThreads - 1) / kAttThreads, bh = B * Hkv;
    const unsigned gy = (unsigned)(bh < 32768 ? bh : 32768);
    e = launch_pdl(attend_score_kernel,
                   dim3((unsigned)(blocks < 1024 ? blocks : 1024), gy, (unsigned)((bh + gy - 1) / gy)),
                   dim3(kAttThreads), 0, st, a, (const float*)logits, (const float*)lse, score_in,
                   score_out);
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}
