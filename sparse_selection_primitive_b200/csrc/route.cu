// Expert routing: the hard top-k of a mixture-of-experts router, its weights
// and the gradient of its logits.  Entry points: lapsum_route and
// lapsum_route_backward (include/lapsum.h).
//
// One warp holds one row of E <= 1024 logits in registers, lane l the
// consecutive experts [l V, (l + 1) V), V = E/32 rounded up to a power of two,
// so that "lowest index first" is "lowest lane first, then lowest slot".  The k-th
// largest of the lanes' best keys bounds the answer from below; the keys that reach it,
// mostly little more than k, are put side by side and ranked by counting.  Where more
// than 32 do (ties), the largest are taken out one by one.
//
// Keys.  Without a bias and groups, the scores rise strictly with the logits,
// so the logits themselves are the keys and the order is exact.  With a bias (or for
// the groups' sums) keys are formed in fp32 with a bound on their error, and a
// row in which two neighbouring ranks lie nearer than that bound is done again
// with fp64 keys, so that the choice is always that of the fp64 keys.  The more ranks, the
// more rows have two that near: softmax keys with a bias, 16384 x 256, take 22 us for 8
// chosen, 91 for 24 and 114 for 32.
//
// What bounds it: instructions, not bytes.  16384 x 256 (8 chosen): 12.1 us for fp32 logits
// (2.8 us of bytes), with 78% of the issue slots taken; 27.6 us for grouped sigmoid keys with
// a bias (1.4 us of bytes).  Taking the largest out one by one, without the bound and the
// ranking of take_largest, made these 18.6 and 60 us.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "elements.cuh"
#include "lapsum_common.cuh"
#include "lapsum_kernels.h"

namespace lapsum {
namespace {

constexpr int kRouteMaxE = 1024;
constexpr int kRouteMaxK = 32;
constexpr int kRouteMaxG = 32;
constexpr int kRouteWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

struct RouteArgs {
    int64_t ld, T;
    int E, k;
    int sigmoid;
    const float* bias;
    int groups, top_groups, group_top;
    int renorm;
    float scale;
    int vec;
    int scratch;  // doubles of shared memory per warp
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
    return x;
}

// This lane's V logits of a row; experts past E read as -inf.
template <class T, int V>
__device__ __forceinline__ void load_lane(const T* row, int E, int lane, bool vec, float out[V]) {
    constexpr int W = V * (int)sizeof(T) <= 16 ? V : 16 / (int)sizeof(T);
    const int base = lane * V;
#pragma unroll
    for (int i = 0; i < V; i += W) {
        if (vec && base + i + W <= E) {
            const Pack<T, W> p = *reinterpret_cast<const Pack<T, W>*>(row + base + i);
#pragma unroll
            for (int j = 0; j < W; ++j) out[i + j] = widen(p.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j)
                out[i + j] = base + i + j < E ? widen(row[base + i + j]) : -INFINITY;
        }
    }
}

// 2^x by the hardware: off by two units, 0 below the smallest normal number
__device__ __forceinline__ float exp2f_near(float x) { return ex2_ftz(x); }
__device__ __forceinline__ float sigmoid_f(float l) { return 1.f / (1.f + expf(-l)); }

// Where expert e of a row lies in the warp's scratch (padded against bank conflicts).
__device__ __forceinline__ int pad_slot(int e) { return e + (e >> 5); }
int pad_size(int E) { return E + (E >> 5) + 1; }

// Key of a group: the sum of its 1 or 2 largest keys; -inf when it has none.  The
// lanes of one group (`sub` consecutive ones) share its experts.
template <class F>
__device__ __forceinline__ F group_score(const F* keys, int size, int g, int groups, int j, int sub,
                                         int group_top) {
    F a = (F)-INFINITY, b = (F)-INFINITY;
    if (g < groups)
        for (int i = j; i < size; i += sub) {
            const F x = keys[pad_slot(g * size + i)];
            if (x > a) {
                b = a;
                a = x;
            } else if (x > b) {
                b = x;
            }
        }
    for (int d = 1; d < sub; d <<= 1) {
        const F a2 = __shfl_xor_sync(kAll, a, d), b2 = __shfl_xor_sync(kAll, b, d);
        const F lo = a < a2 ? a : a2, hi = a < a2 ? a2 : a;
        const F m = b < b2 ? b2 : b;
        a = hi;
        b = lo < m ? m : lo;
    }
    return group_top == 2 && b > (F)-INFINITY ? a + b : a;
}

// Whether this lane's group g (value `mine`; `sub` lanes each) is among the `top` best
// of all by (value, lowest index).  *gap gets the distance between the last kept and the
// first dropped value (+inf where nothing is dropped).
template <class F>
__device__ __forceinline__ bool kept_here(F mine, int g, int groups, int sub, int top, F* gap) {
    int rank = 0;
    for (int o = 0; o < groups; ++o) {
        const F x = __shfl_sync(kAll, mine, o * sub);
        if (x > mine || (x == mine && o < g)) ++rank;
    }
    const bool real = g < groups && mine > (F)-INFINITY;
    const bool keep = real && rank < top;
    F lo = keep ? mine : (F)INFINITY, hi = real && !keep ? mine : (F)-INFINITY;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const F l2 = __shfl_xor_sync(kAll, lo, d), h2 = __shfl_xor_sync(kAll, hi, d);
        lo = l2 < lo ? l2 : lo;
        hi = h2 > hi ? h2 : hi;
    }
    *gap = hi > (F)-INFINITY && lo < (F)INFINITY ? lo - hi : (F)INFINITY;
    return keep;
}
__device__ __forceinline__ unsigned group_mask(bool keep, int groups, int sub) {
    const unsigned lanes = __ballot_sync(kAll, keep);
    unsigned mask = 0;
    for (int o = 0; o < groups; ++o) mask |= ((lanes >> (o * sub)) & 1u) << o;
    return mask;
}

// What fp64 keys of a row take beside its own logit: nothing, or (softmax) the largest
// logit and the sum of e^{l - m}.
struct RowSum {
    double m, total;
};
template <class T>
__device__ __forceinline__ RowSum row_sum_fp64(const T* row, const RouteArgs& a, int lane) {
    RowSum s{0.0, 1.0};
    if (a.sigmoid) return s;
    s.m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) s.m = fmax(s.m, (double)widen(row[e]));
#pragma unroll
    for (int d = 16; d; d >>= 1) s.m = fmax(s.m, __shfl_xor_sync(kAll, s.m, d));
    s.total = 0.0;
    for (int e = lane; e < a.E; e += 32) s.total += exp((double)widen(row[e]) - s.m);
#pragma unroll
    for (int d = 16; d; d >>= 1) s.total += __shfl_xor_sync(kAll, s.total, d);
    return s;
}
template <class T>
__device__ __forceinline__ double key_fp64(const T* row, const RouteArgs& a, int e, RowSum s) {
    const double l = (double)widen(row[e]);
    double c = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - s.m) / s.total;
    if (a.bias != nullptr) c += (double)a.bias[e];
    return l == -INFINITY ? -INFINITY : c;
}

// The order of `found` <= 32 candidates (lane c holds expert e) by their fp64 keys: the
// j-th expert comes back on lane j.
template <class T>
__device__ __noinline__ int rank_fp64(const T* row, const RouteArgs& a, int lane, int e, int found) {
    const RowSum s = row_sum_fp64(row, a, lane);
    const double mine = lane < found ? key_fp64(row, a, e, s) : -INFINITY;
    int rank = 0;
    for (int c = 0; c < found; ++c) {
        const double x = __shfl_sync(kAll, mine, c);
        const int o = __shfl_sync(kAll, e, c);
        rank += (x > mine || (x == mine && o < e)) ? 1 : 0;
    }
    int at = -1;
    for (int c = 0; c < found; ++c) {
        const int r = __shfl_sync(kAll, rank, c), o = __shfl_sync(kAll, e, c);
        if (r == lane) at = o;
    }
    return at;
}

// The choice with fp64 keys, from the logits in memory: the j-th chosen expert
// is returned on lane j (-1: none).  `keys` is the warp's scratch.
template <class T>
__device__ __noinline__ int route_row_fp64(const T* row, const RouteArgs& a, int lane,
                                           double* keys) {
    const RowSum s = row_sum_fp64(row, a, lane);
    __syncwarp();
    for (int e = lane; e < a.E; e += 32) keys[pad_slot(e)] = key_fp64(row, a, e, s);
    __syncwarp();
    unsigned kept = kAll;
    const int size = a.E / a.groups;
    if (a.groups > 1) {
        int gp = 1;
        while (gp < a.groups) gp <<= 1;
        const int sub = 32 / gp, g = lane / sub;
        const double mine =
            group_score<double>(keys, size, g, a.groups, lane % sub, sub, a.group_top);
        double gap;
        kept = group_mask(kept_here<double>(mine, g, a.groups, sub, a.top_groups, &gap), a.groups,
                          sub);
    }
    int chosen = -1;
    for (int j = 0; j < a.k; ++j) {
        double best = -INFINITY;
        int at = a.E;
        for (int e = lane; e < a.E; e += 32)
            if ((kept >> (a.groups > 1 ? e / size : 0)) & 1u) {
                const double x = keys[pad_slot(e)];
                // without a bias the logits break ties of keys that round to the same
                const bool better =
                    x > best || (x == best && at < a.E && a.bias == nullptr &&
                                 widen(row[e]) > widen(row[at]));
                if (better) {
                    best = x;
                    at = e;
                }
            }
        float lb = at < a.E ? widen(row[at]) : -INFINITY;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const double x = __shfl_xor_sync(kAll, best, d);
            const int o = __shfl_xor_sync(kAll, at, d);
            const float lo = __shfl_xor_sync(kAll, lb, d);
            const bool up = a.bias == nullptr && lo != lb ? lo > lb : o < at;
            if (x > best || (x == best && up)) {
                best = x;
                at = o;
                lb = lo;
            }
        }
        if (!(best > -INFINITY)) break;
        if (lane == j) chosen = at;
        __syncwarp();
        if (lane == 0) keys[pad_slot(at)] = -INFINITY;
        __syncwarp();
    }
    return chosen;
}

// Scores to within the bound below; __fdividef and ex2 are approximations of the hardware.
__device__ __forceinline__ float near_sigmoid(float l) {
    return __fdividef(1.f, 1.f + exp2f_near(-l * kLog2e));
}

// The largest keys of a row in order, ties by the lower index: lane j gets the j-th one's
// expert (-1: none) and key (0), for `count` lanes at least.  Every lane offers its largest key, and the
// count-th largest offer bounds the answer from below; the keys that reach it, mostly
// little more than `count`, are put side by side and ranked by counting.  Too many of them
// (ties): the largest are taken out one by one.  Returns how many lanes hold one when those
// are all keys from *bound on, else 0.
template <int V>
__device__ __forceinline__ int take_largest(uint32_t (&key)[V], int count, int lane, uint2* cand,
                                            int* chosen, uint32_t* chosen_key, uint32_t* reach) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    uint32_t offer = best, bound = 1;
    for (int j = 0; j < count; ++j) {
        const uint32_t top = __reduce_max_sync(kAll, offer);
        bound = top;
        if (top == 0u) break;
        if (offer == top) offer = 0;
    }
    bound = max(bound, 1u);
    const unsigned below = (1u << lane) - 1u;
    int found = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const bool in = key[i] >= bound;
        const unsigned who = __ballot_sync(kAll, in);
        const int at = found + __popc(who & below);
        if (in && at < 32) cand[at] = make_uint2(key[i], (uint32_t)(lane * V + i));
        found += __popc(who);
    }
    *chosen = -1;
    *chosen_key = 0;
    if (found <= 32) {
        __syncwarp();
        const uint2 mine = lane < found ? cand[lane] : make_uint2(0u, 0u);
        int rank = 0;
        for (int c = 0; c < found; ++c) {
            const uint2 o = cand[c];
            rank += (o.x > mine.x || (o.x == mine.x && o.y < mine.y)) ? 1 : 0;
        }
        __syncwarp();
        if (lane < found) cand[rank] = mine;
        __syncwarp();
        if (lane < found) {
            *chosen = (int)cand[lane].y;
            *chosen_key = cand[lane].x;
        }
        *reach = bound;
        return found;
    }
    for (int j = 0; j < count; ++j) {
        const uint32_t top = __reduce_max_sync(kAll, best);
        if (top == 0u) break;
        const int src = __ffs(__ballot_sync(kAll, best == top)) - 1;
        int at = 0;
        if (lane == src) {
            bool done = false;
            best = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!done && key[i] == top) {
                    done = true;
                    at = lane * V + i;
                    key[i] = 0;
                }
                best = max(best, key[i]);
            }
        }
        at = __shfl_sync(kAll, at, src);
        if (lane == j) {
            *chosen = at;
            *chosen_key = top;
        }
    }
    return 0;
}

// One warp per row.  kKeyed: keys are scores (+ bias) or groups limit the choice;
// otherwise the logits are the keys.
template <class T, int V, bool kKeyed>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_kernel(const T* logits, RouteArgs a, float* weights, int32_t* experts) {
    pdl_wait();
    extern __shared__ double route_scratch[];
    __shared__ uint2 candidates[kRouteWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const T* row = logits + t * a.ld;
    float l[V];
    load_lane<T, V>(row, a.E, lane, a.vec != 0, l);

    bool bad = false;  // a NaN or +inf anywhere makes the row's answer NaN
#pragma unroll
    for (int i = 0; i < V; ++i) bad |= !(l[i] < INFINITY);

    float m = 0.f, total = 0.f;  // softmax: the largest logit, the sum of e^{l - m}
    if (!a.sigmoid && (kKeyed || !a.renorm)) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
        m = warp_max(m);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += l[i] == -INFINITY ? 0.f : exp2f_near((l[i] - m) * kLog2e);
        total = warp_sum(s);
    }

    uint32_t key[V];  // 0: not to be chosen (no finite value has that key)
    bool near = false;
    float tol = 0.f;
    if constexpr (kKeyed) {
        float* fs = reinterpret_cast<float*>(route_scratch + (size_t)warp * a.scratch);
        const float inv = total > 0.f ? 1.f / total : 0.f;
        float c[V];
        float cmax = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            c[i] = -INFINITY;
            if (l[i] > -INFINITY) {
                float x = a.sigmoid ? near_sigmoid(l[i]) : exp2f_near((l[i] - m) * kLog2e) * inv;
                if (a.bias != nullptr) x += a.bias[e];
                bad |= !(x < INFINITY);
                c[i] = x;
                if (x > -INFINITY) cmax = fmaxf(cmax, fabsf(x));
            }
        }
        // How far a key may be off.  Sigmoid: e^-l is off by (|l| + 4) 2^-24 relative, which
        // s (1 - s) brings below 1.3 units, the sum and the quotient by three more.  Softmax:
        // 2 |l - m| + 4 units in the numerator, the same on average and V + 5 more in the
        // sum, all relative to a score of at most 1 / sum.  The bias adds a rounding.
        cmax = warp_max(cmax);
        tol = 5.97e-8f * ((a.sigmoid ? 8.f : 64.f * inv) + 2.f * cmax);
        bool kept = true;           // this lane's experts are in a kept group
        unsigned kept_mask = kAll;  // or which groups are
        const int size = a.E / a.groups;
        // lanes per group, where its experts are whole lanes and a power of two of them
        const int span = size % V == 0 && ((size / V) & (size / V - 1)) == 0 ? size / V : 0;
        if (a.groups > 1) {
            float gap;
            if (span > 0) {
                float u = -INFINITY, w = -INFINITY;  // the group's two largest keys
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    w = fmaxf(w, fminf(u, c[i]));
                    u = fmaxf(u, c[i]);
                }
                for (int d = 1; d < span; d <<= 1) {
                    const float u2 = __shfl_xor_sync(kAll, u, d), w2 = __shfl_xor_sync(kAll, w, d);
                    w = fmaxf(fminf(u, u2), fmaxf(w, w2));
                    u = fmaxf(u, u2);
                }
                const float mine = a.group_top == 2 && w > -INFINITY ? u + w : u;
                kept = kept_here<float>(mine, lane / span, a.groups, span, a.top_groups, &gap);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (lane * V + i < a.E) fs[pad_slot(lane * V + i)] = c[i];
                __syncwarp();
                int gp = 1;
                while (gp < a.groups) gp <<= 1;
                const int sub = 32 / gp, g = lane / sub;
                const float mine =
                    group_score<float>(fs, size, g, a.groups, lane % sub, sub, a.group_top);
                const bool keep = kept_here<float>(mine, g, a.groups, sub, a.top_groups, &gap);
                kept_mask = group_mask(keep, a.groups, sub);
                __syncwarp();
            }
            near |= gap <= 5.f * tol;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool in = c[i] > -INFINITY && kept &&
                            (kept_mask == kAll || ((kept_mask >> ((lane * V + i) / size)) & 1u));
            // -0 and +0 are one value
            key[i] = in ? to_key((a.bias != nullptr ? c[i] : l[i]) + 0.f) : 0u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = l[i] > -INFINITY ? to_key(l[i] + 0.f) : 0u;
    }
    bad = __any_sync(kAll, bad);

    int chosen;
    uint32_t mine, reach = 0;
    // with a bias more ranks are looked at: the chosen set ends between two keys
    const bool check = kKeyed && a.bias != nullptr;
    const int found = take_largest<V>(key, check ? min(a.k + 2, 32) : a.k, lane, candidates[warp],
                                      &chosen, &mine, &reach);
    if constexpr (kKeyed) {
        bool close = false;  // two neighbouring ranks that fp32 does not tell apart
        if (check) {
            uint32_t next = __shfl_down_sync(kAll, mine, 1);
            if (a.k == 32) {  // no lane holds the key after the last one: the largest that is left
                uint32_t left = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (found == 0 || key[i] < reach) left = max(left, key[i]);
                reach = __reduce_max_sync(kAll, left);
                if (lane == 31) next = reach;
            }
            close = lane < a.k && mine != 0u && next != 0u &&
                    from_key(mine) - from_key(next) <= 2.f * tol;
            close = __any_sync(kAll, close);
        }
        near = __any_sync(kAll, near);  // or two groups
        if (close && !near && !bad) {
            // all that may belong to the first k are among the candidates when those reach
            // further than the error below the k-th
            const uint32_t kth = __shfl_sync(kAll, mine, a.k - 1);
            if (found > 0 && (kth == 0u || reach <= 1u ||
                              from_key(kth) - 2.f * tol > from_key(reach)))
                chosen = rank_fp64<T>(row, a, lane, chosen, found);
            else
                near = true;
        }
    }
    if constexpr (kKeyed) {
        if (near && !bad)
            chosen = route_row_fp64<T>(row, a, lane, route_scratch + (size_t)warp * a.scratch);
    }
    if (lane >= a.k) chosen = -1;

    // weights: lane j owns the j-th choice
    float w = 0.f;
    const float lc = chosen >= 0 ? widen(row[chosen]) : -INFINITY;
    if (a.renorm) {
        const float lm = warp_max(lc);
        // softmax: the sum over all experts cancels, leaving a softmax over the
        // chosen ones.  Sigmoids that are all below e^-60 equal e^l to fp32, so
        // the same form keeps their ratio where they would underflow.
        const bool expform = !a.sigmoid || lm < -60.f;
        const float s = chosen < 0 ? 0.f : expform ? expf(lc - lm) : sigmoid_f(lc);
        const float sum = warp_sum(s);
        w = chosen < 0 ? 0.f : s / sum * a.scale;
    } else if (chosen >= 0) {
        w = (a.sigmoid ? sigmoid_f(lc) : expf(lc - m) / total) * a.scale;
    }
    if (bad) {
        chosen = -1;
        w = NAN;
    }
    if (lane < a.k) {
        weights[t * a.k + lane] = w;
        experts[t * a.k + lane] = chosen;
    }
}

// Gradient of the logits.  With s the scores, w the weights and u = dL/dw, sums over the chosen:
//   renormalised: d_i = w_i sum_j (w_j / scale) (u_i - u_j) on the chosen experts
//                 (softmax), times 1 - s_i (sigmoid), 0 elsewhere;
//   softmax:      d_i = s_i (scale u_i rest + sum_j w_j (u_i - u_j)) on the chosen experts,
//                 rest the sum of the others' scores, and -s_i sum_j u_j w_j elsewhere;
//   sigmoid:      d_i = u_i w_i (1 - s_i) on the chosen experts.
// The sums are of differences: u_i - sum_j u_j w_j / scale is the same number, but where one
// weight dominates it cancels to what the others leave (6% off when they are e^-16 of it).
// With W the sum of the w_j and 0 the expert of the largest,
//     sum_j w_j (u_i - u_j) = W (u_i - u_0) - sum_j w_j (u_j - u_0),
// one sum for all i: for i = 0 the dominating term is exactly 0, and as w_0 >= W / k, the two
// parts are at most 2 k + 1 times the sum of magnitudes for any i.
// A row whose weights are NaN gets NaN.  9.0 us for 16384 x 256 fp32 (2.8 us of bytes); carrying
// the chosen terms to the lanes that own their experts instead of storing them on top took 19.
template <class T, int V>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_backward_kernel(const T* logits, RouteArgs a, const float* weights,
                          const int32_t* experts, const float* dw, T* out, int64_t ld_out,
                          int vec_out) {
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const T* row = logits + t * a.ld;
    int e = -1;
    float w = 0.f, u = 0.f;
    bool bad = false;
    if (lane < a.k) {
        e = experts[t * a.k + lane];
        w = weights[t * a.k + lane];
        bad = isnan(w);
        if (e >= a.E) e = -1;
        if (e >= 0) u = dw[t * a.k + lane];
    }
    bad = __any_sync(kAll, bad);
    const bool dense = !a.sigmoid && !a.renorm;
    const float share = e < 0 ? 0.f : a.renorm ? w / a.scale : w;
    const float le = e >= 0 && (dense || a.sigmoid) ? widen(row[e]) : 0.f;
    float apart = 0.f;  // sum of share_j (u_i - u_j)
    if (dense || a.renorm) {
        // shares are not negative, so that their order is that of their words
        const uint32_t most = __reduce_max_sync(kAll, __float_as_uint(share));
        const int top = __ffs(__ballot_sync(kAll, __float_as_uint(share) == most)) - 1;
        const float from = u - __shfl_sync(kAll, u, top);
        const float all = dense ? warp_sum(share) : 1.f;
        apart = fmaf(all, from, -warp_sum(e < 0 ? 0.f : share * from));
    }
    // every expert's gradient but for the chosen ones' own terms; those follow on top
    float d[V];
    float score = 0.f, rest = 0.f;  // dense: of the lane's chosen expert, of all that are not chosen
    if (dense) {
        const float dot = warp_sum(share * u);
        __shared__ unsigned marks[kRouteWarps][32];
        marks[warp][lane] = 0;
        __syncwarp();
        if (e >= 0) atomicOr(&marks[warp][e / V], 1u << (e % V));
        float l[V];
        load_lane<T, V>(row, a.E, lane, a.vec != 0, l);
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
        m = warp_max(m);
        __syncwarp();
        const unsigned chosen = marks[warp][lane];  // which of this lane's V experts
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            d[i] = l[i] == -INFINITY ? 0.f : exp2f_near((l[i] - m) * kLog2e);
            s += d[i];
            rest += (chosen >> i) & 1u ? 0.f : d[i];
        }
        s = warp_sum(s);
        const float inv = s > 0.f ? 1.f / s : 0.f;
        rest = warp_sum(rest) * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = d[i] == 0.f ? 0.f : d[i] * inv * -dot;
        if (e >= 0) score = expf(le - m) * inv;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = 0.f;
    }
    if (bad) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = NAN;
    }
    constexpr int W = V * (int)sizeof(T) <= 16 ? V : 16 / (int)sizeof(T);
    T* o = out + t * ld_out;
    const int first = lane * V;
#pragma unroll
    for (int i = 0; i < V; i += W) {
        if (vec_out && first + i + W <= a.E) {
            Pack<T, W> p;
#pragma unroll
            for (int j = 0; j < W; ++j) p.v[j] = narrow<T>(d[i + j]);
            *reinterpret_cast<Pack<T, W>*>(o + first + i) = p;
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (first + i + j < a.E) o[first + i + j] = narrow<T>(d[i + j]);
        }
    }
    __syncwarp();  // orders the row's stores before the chosen experts' own
    if (e < 0 || bad) return;
    float own = dense ? score * fmaf(a.scale * rest, u, apart) : w * (a.renorm ? apart : u);
    if (a.sigmoid) own *= sigmoid_f(-le);  // 1 - s
    o[e] = narrow<T>(own);
}

int lane_values(int E) {
    int v = 1;
    while (v * 32 < E) v <<= 1;
    return v;
}

template <class F>
cudaError_t with_lane_values(int E, F f) {
    switch (lane_values(E)) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 8: return f(std::integral_constant<int, 8>{});
        case 16: return f(std::integral_constant<int, 16>{});
        default: return f(std::integral_constant<int, 32>{});
    }
}

// Whether a lane's V elements can be moved as 16-byte (or shorter) packs.
bool lane_packs(const void* p, int64_t ld, int E, int size) {
    const int v = lane_values(E), w = v * size <= 16 ? v : 16 / size;
    return aligned_to(p, (size_t)w * size) && ld % w == 0;
}

bool route_sizes_ok(int64_t ld, int64_t T, int64_t E, int32_t k, int score, float scale) {
    return T >= 1 && T <= (int64_t(1) << 31) && E >= 1 && E <= kRouteMaxE && k >= 1 &&
           k <= kRouteMaxK && k <= E && ld >= E &&
           (score == LAPSUM_SCORE_SOFTMAX || score == LAPSUM_SCORE_SIGMOID) && scale > 0.f &&
           std::isfinite(scale);
}

}  // namespace
}  // namespace lapsum

using namespace lapsum;

extern "C" int lapsum_route(const void* logits, int dtype, int64_t ld, int64_t T, int64_t E,
                            int32_t k, int score, const float* bias, int32_t groups,
                            int32_t top_groups, int32_t group_top, int renormalize, float scale,
                            float* weights, int32_t* experts, void* stream) {
    if (logits == nullptr || weights == nullptr || experts == nullptr) return LAPSUM_EINVAL;
    if (!known_dtype(dtype) || !route_sizes_ok(ld, T, E, k, score, scale)) return LAPSUM_EINVAL;
    if (groups < 1 || groups > kRouteMaxG || E % groups != 0 || top_groups < 1 ||
        top_groups > groups || (group_top != 1 && group_top != 2))
        return LAPSUM_EINVAL;
    if (k > top_groups * (E / groups)) return LAPSUM_EINVAL;
    if (!aligned_to(logits, dtype_size(dtype)) || !aligned_to(weights, 4) ||
        !aligned_to(experts, 4) || !aligned_to(bias, 4))
        return LAPSUM_EINVAL;
    // keeping every group limits nothing
    const int g = top_groups == groups ? 1 : groups;
    RouteArgs a{ld, T, (int)E, k, score == LAPSUM_SCORE_SIGMOID, bias, g, g == 1 ? 1 : top_groups,
                group_top, renormalize != 0, scale,
                lane_packs(logits, ld, (int)E, dtype_size(dtype)) ? 1 : 0,
                pad_size((int)E)};
    cudaStream_t st = (cudaStream_t)stream;
    const dim3 grid((unsigned)((T + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
    ProfScope prof("route", st);
    const cudaError_t e = with_dtype(dtype, [&](auto* tag) {
        using T_ = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        return with_lane_values((int)E, [&](auto v) {
            constexpr int V = decltype(v)::value;
            if (bias != nullptr || g > 1)
                return launch_pdl(route_kernel<T_, V, true>, grid, block,
                                  (size_t)kRouteWarps * a.scratch * sizeof(double), st,
                                  (const T_*)logits, a, weights, experts);
            return launch_pdl(route_kernel<T_, V, false>, grid, block, 0, st, (const T_*)logits, a,
                              weights, experts);
        });
    });
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}

extern "C" int lapsum_route_backward(const void* logits, int dtype, int64_t ld, int64_t T,
                                     int64_t E, int32_t k, int score, int renormalize, float scale,
                                     const float* weights, const int32_t* experts,
                                     const float* dweights, void* dlogits, int64_t ld_out,
                                     void* stream) {
    if (logits == nullptr || weights == nullptr || experts == nullptr || dweights == nullptr ||
        dlogits == nullptr)
        return LAPSUM_EINVAL;
    if (!known_dtype(dtype) || !route_sizes_ok(ld, T, E, k, score, scale) || ld_out < E)
        return LAPSUM_EINVAL;
    const int size = dtype_size(dtype);
    if (!aligned_to(logits, size) || !aligned_to(dlogits, size) || !aligned_to(weights, 4) ||
        !aligned_to(experts, 4) || !aligned_to(dweights, 4))
        return LAPSUM_EINVAL;
    RouteArgs a{ld, T, (int)E, k, score == LAPSUM_SCORE_SIGMOID, nullptr, 1, 1, 1,
                renormalize != 0, scale, lane_packs(logits, ld, (int)E, size) ? 1 : 0, 0};
    const int vec_out = lane_packs(dlogits, ld_out, (int)E, size) ? 1 : 0;
    cudaStream_t st = (cudaStream_t)stream;
    const dim3 grid((unsigned)((T + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
    ProfScope prof("route_backward", st);
    const cudaError_t e = with_dtype(dtype, [&](auto* tag) {
        using T_ = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        return with_lane_values((int)E, [&](auto v) {
            constexpr int V = decltype(v)::value;
            return launch_pdl(route_backward_kernel<T_, V>, grid, block, 0, st, (const T_*)logits,
                              a, weights, experts, dweights, (T_*)dlogits, ld_out, vec_out);
        });
    });
    return e == cudaSuccess ? LAPSUM_OK : LAPSUM_ECUDA;
}
