// Mixture of experts around the experts' products (sq_fp8b.cuh): choice of the
// experts (route), the rows' order by expert (dispatch) and the weighted sum of
// a token's expert outputs (combine).
#pragma once

#include <cuda_bf16.h>

#include "sq_device.cuh"

namespace sqm {

constexpr int MAX_EXPERTS = 512;
constexpr int MAX_TOP = 16;
constexpr int MAX_GROUPS = 32;
constexpr int RT_WARPS = 4;

// ---------------------------------------------------------------- route
// p = softmax or sigmoid of a token's logits; an expert's score is p + bias
// (the logit itself where that gives the same order: no bias, and groups
// judged by one score); the best `keep` of `groups` equal groups by the sum of
// their group_top best scores, then the `top` best scores inside them, ties to
// the lower index.  Weights: p at the chosen experts, over their sum + 1e-20
// if renorm, times scale.  A logit of -inf or NaN is never chosen (+inf counts
// as the largest finite value); missing choices are -1 with weight 0.
//
// The order is that of the scores in 64 bits.  They are computed in fp32
// first; where two scores that decide something are closer than the fp32
// error, the warp does the token again in fp64.  Scores that are logits
// are exact and never need it.
//
// One warp per token, expert e in lane e % 32.  A choice is one integer
// maximum over the warp (order-preserving keys) and one minimum for the index.
struct RouteArgs {
    const void *logits;
    int64_t T, ld;
    const float *bias;
    int E, top, groups, keep, group_top;
    int bf16, sigmoid, renorm;
    float scale;
    int32_t *ids;
    float *weights;
};

// Order-preserving unsigned keys; 0 is below every finite score.
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t u = __float_as_uint(v);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(double v)
{
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
    return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }
__device__ __forceinline__ double value_of(uint64_t k)
{
    return __longlong_as_double(static_cast<long long>(k ^ ((k >> 63) ? 0x8000000000000000ull : ~0ull)));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(0xFFFFFFFFu, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k)
{
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

__device__ __forceinline__ float exp_t(float v) { return expf(v); }
__device__ __forceinline__ double exp_t(double v) { return exp(v); }

template <typename T>
__device__ __forceinline__ T warp_sum(T v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// A score closer than this to another one decides nothing in fp32 (relative to
// the larger of 1 and the score): exponentials, the sum of up to 512 of them, the
// quotient and the bias leave less than 2^-18.
__device__ __forceinline__ bool too_close(float a, float b) { return a - b <= 7.62939453125e-6f * fmaxf(1.0f, fmaxf(fabsf(a), fabsf(b))); }
__device__ __forceinline__ bool too_close(double, double) { return false; }

__device__ __forceinline__ float load_logit(const RouteArgs &a, int64_t t, int e)
{
    const float l = a.bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(a.logits)[t * a.ld + e]) << 16)
                           : static_cast<const float *>(a.logits)[t * a.ld + e];
    return l != l ? -INFINITY : fminf(l, 3.402823466e38f);
}

// Chosen experts of one token: lane j < top holds the j-th (-1: none).  Returns
// false (all lanes) where fp32 scores cannot decide.  stat receives what p needs:
// the largest logit and the sum of exponentials (softmax).
template <typename T, int V>
__device__ __forceinline__ bool choose(const RouteArgs &a, const float (&l)[V], bool by_logit, int lane, int &mine, float &lmax, T &sum)
{
    using Key = decltype(key_of(T()));
    if (!a.sigmoid) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) mx = fmaxf(mx, l[i]);
        lmax = value_of(warp_max(key_of(mx)));
        T s = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) s += l[i] == -INFINITY ? T(0) : exp_t(static_cast<T>(l[i]) - static_cast<T>(lmax));
        sum = warp_sum(s);
    }
    Key key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        T v = static_cast<T>(l[i]);
        if (!by_logit) {
            v = a.sigmoid ? T(1) / (T(1) + exp_t(-v)) : exp_t(v - static_cast<T>(lmax)) / sum;
            if (a.bias && e < a.E) v += static_cast<T>(a.bias[e]);
        }
        key[i] = l[i] == -INFINITY ? Key(0) : key_of(v);
    }
    bool sure = true;
    if (a.groups > 1) {
        const int per = a.E / a.groups;
        Key gkey = 0;   // lane g: group g's worth
        for (int g = 0; g < a.groups; ++g) {
            T worth = 0;
            bool some = false;
            int skip = -1;
            for (int n = 0; n < a.group_top; ++n) {
                Key best = 0;
                int at = 0x7FFFFFFF;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = lane + 32 * i;
                    if (e >= g * per && e < (g + 1) * per && e != skip && key[i] > best) { best = key[i]; at = e; }
                }
                const Key top = warp_max(best);
                if (top == 0) break;
                skip = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(best == top ? at : 0x7FFFFFFF)));
                worth += value_of(top);
                some = true;
            }
            if (lane == g) gkey = some ? key_of(worth) : Key(0);
        }
        uint32_t open = 0;
        T last = 0;
        for (int n = 0; n <= a.keep && n < a.groups; ++n) {
            const Key best = warp_max((open >> lane) & 1u ? Key(0) : gkey);
            if (best == 0) break;
            const T v = value_of(best);
            if (n == a.keep) {
                if (!by_logit && too_close(last, v)) sure = false;
                break;
            }
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, !((open >> lane) & 1u) && gkey == best);
            open |= who & (0u - who);
            last = v;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((open >> (e / per)) & 1u)) key[i] = 0;
        }
    }
    mine = -1;
    T last = 0;
    for (int n = 0; n <= a.top; ++n) {
        Key best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) { best = key[i]; at = lane + 32 * i; }
        const Key top = warp_max(best);
        if (top == 0) break;
        const T v = value_of(top);
        if (n > 0 && !by_logit && too_close(last, v)) sure = false;
        if (n == a.top) break;
        const int e = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(best == top ? at : 0x7FFFFFFF)));
        if (lane == n) mine = e;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == lane + 32 * i) key[i] = 0;
        last = v;
    }
    return sure;
}

template <int V>
__global__ void __launch_bounds__(32 * RT_WARPS) route_kernel(const RouteArgs a)
{
    sqd::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
    sqd::pdl_wait();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * RT_WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;
    float l[V];
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = lane + 32 * i < a.E ? load_logit(a, t, lane + 32 * i) : -INFINITY;
    int mine;
    float lmax = 0.0f, sum = 1.0f;
    if (!choose<float, V>(a, l, by_logit, lane, mine, lmax, sum)) {
        double sum64 = 1.0;
        choose<double, V>(a, l, by_logit, lane, mine, lmax, sum64);
    }
    float p = 0.0f;
    if (mine >= 0) {
        const float v = load_logit(a, t, mine);
        p = a.sigmoid ? 1.0f / (1.0f + expf(-v)) : expf(v - lmax) / sum;
    }
    if (a.renorm) p /= warp_sum(p) + 1e-20f;
    if (lane < a.top) {
        a.ids[t * a.top + lane] = mine;
        a.weights[t * a.top + lane] = p * a.scale;
    }
}

// ---------------------------------------------------------------- dispatch
// Order of the (token, choice) pairs by expert, stable: pos[i] = row of pair i
// (its expert's offset plus the pairs of the same expert before it), -1 for an
// index outside [0, E); offsets[E + 1].  One CTA: warp w owns a contiguous
// range of pairs, counts its experts, and after a scan over warps and experts
// gives out rows in order, 32 pairs at a time (lanes with the same expert rank
// themselves by lane).  No atomics decide an order.
constexpr int DP_WARPS = 32;

__global__ void __launch_bounds__(32 * DP_WARPS) dispatch_kernel(const int32_t *__restrict__ ids, int64_t pairs, int E,
                                                                 int32_t *__restrict__ offsets, int32_t *__restrict__ pos)
{
    extern __shared__ int32_t cnt[];   // [DP_WARPS][E], then [E + 1] offsets
    int32_t *off = cnt + DP_WARPS * E;
    sqd::pdl_launch_dependents();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < DP_WARPS * E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    sqd::pdl_wait();
    const int64_t per = ((pairs + DP_WARPS - 1) / DP_WARPS + 31) / 32 * 32;
    const int64_t lo = min(per * w, pairs), hi = min(lo + per, pairs);
    int32_t *mine = cnt + w * E;
    for (int64_t i = lo + lane; i < hi; i += 32) {
        const int e = ids[i];
        if (e >= 0 && e < E) atomicAdd(mine + e, 1);
    }
    __syncthreads();
    // counts -> first row of every (warp, expert), relative to the expert
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int32_t s = 0;
        for (int v = 0; v < DP_WARPS; ++v) {
            const int32_t c = cnt[v * E + e];
            cnt[v * E + e] = s;
            s += c;
        }
        off[e + 1] = s;
    }
    __syncthreads();
    if (w == 0) {   // inclusive scan of the experts' totals
        int32_t base = 0;
        if (lane == 0) off[0] = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            int32_t v = e < E ? off[e + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o) v += u;
            }
            if (e < E) off[e + 1] = base + v;
            base += __shfl_sync(0xFFFFFFFFu, v, 31);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = off[e];
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        const int64_t i = i0 + lane;
        int e = i < hi ? ids[i] : -1;
        if (e < 0 || e >= E) e = -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int32_t r = -1;
        if (e >= 0) r = off[e] + mine[e] + rank;
        __syncwarp();
        if (e >= 0 && rank == 0) mine[e] += __popc(same);
        __syncwarp();
        if (i < hi) pos[i] = r;
    }
}

// ---------------------------------------------------------------- combine
// Y[t] = sum_j weights[t, j] Z[pos[t, j]] over the choices that have a row, in
// the order of j, fp32, rounded once.  One thread per 8 columns; the rows of Z
// that have no choice are never read.  Memory-bound: top + 1 rows of 2 N bytes.
constexpr int CB_THREADS = 256;

__global__ void __launch_bounds__(CB_THREADS) combine_kernel(const uint16_t *__restrict__ Z, int64_t rows_z, int64_t ldz,
                                                             const int32_t *__restrict__ pos, const float *__restrict__ weights,
                                                             int64_t T, int top, int N, uint16_t *__restrict__ Y, int64_t ldy)
{
    sqd::pdl_launch_dependents();
    sqd::pdl_wait();
    const int per = N >> 3;
    const int64_t total = T * per;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * CB_THREADS + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * CB_THREADS) {
        const int64_t t = i / per;
        const int c = static_cast<int>(i - t * per) * 8;
        float acc[8] = {};
        for (int j = 0; j < top; ++j) {
            const int64_t r = pos[t * top + j];
            if (r < 0 || r >= rows_z) continue;
            const float w = weights[t * top + j];
            const uint4 v = *reinterpret_cast<const uint4 *>(Z + r * ldz + c);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                acc[2 * q] = fmaf(w, __uint_as_float(u[q] << 16), acc[2 * q]);
                acc[2 * q + 1] = fmaf(w, __uint_as_float(u[q] & 0xFFFF0000u), acc[2 * q + 1]);
            }
        }
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * q], acc[2 * q + 1]);
            o[q] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(Y + t * ldy + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace sqm
