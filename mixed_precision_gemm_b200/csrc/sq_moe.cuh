// Mixture of experts around the experts' products (sq_fp8b.cuh): choice of the
// experts (route), the rows' order by expert (dispatch) and the weighted sum of
// a token's expert outputs (combine).
#pragma once

#include <cuda_bf16.h>

#include "sq_device.cuh"
#include "sq_fp8b.cuh"

namespace sqm {

constexpr int MAX_EXPERTS = 512;
constexpr int MAX_TOP = 16;
constexpr int MAX_GROUPS = 32;
constexpr int RT_WARPS = 4;

// ---------------------------------------------------------------- route
// p = softmax or sigmoid of a token's logits; an expert's score is p + bias
// (the logit itself where p need not be known: no bias, and groups judged by one
// score; it also orders values of p that are the same number); the best `keep` of `groups` equal groups by the sum of
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
// One warp per token, V = E / 32 rounded up to a power of two consecutive experts
// per lane.  A choice is one integer maximum over the warp (order-preserving keys)
// and a ballot for the lowest lane that has it.
struct RouteArgs {
    const void *logits;
    int64_t T, ld;
    const float *bias;
    int E, top, groups, keep, group_top;
    int bf16, sigmoid, renorm, vec;
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

template <typename T>
__device__ __forceinline__ T warp_sum(T v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Two scores whose fp32 values are this close (size: the larger magnitude) are put in
// order in fp64.  A score is off by less than 20 u + 2^-24 |score|, u = 2^-23: of a softmax
// value p = e^-x / S the exponential (2 u and 1.2 u x, its argument's rounding 0.5 u x; times
// p at most 2 u), the sum's terms (at most 4 u times p for up to 512 of them), its up to 20
// additions (10 u) and the quotient (2.5 u); of a sigmoid value 4 u; half a step for the bias.
// The two sides of a comparison come to 41 u max(1, size), taken as 64 u = 2^-17.
// A group's sum of two scores has the errors of both, and the rounding of the sum,
// however small it is: size is then twice max(1, the sum of their magnitudes).
__device__ __forceinline__ bool too_close(float a, float b, float size) { return a - b <= 7.62939453125e-6f * fmaxf(1.0f, size); }
__device__ __forceinline__ bool too_close(double, double, float) { return false; }

// (-0 + 0 is +0: the keys of the two zeros differ, and they are a tie)
__device__ __forceinline__ float finite_logit(float l) { return l != l ? -INFINITY : fminf(l, 3.402823466e38f) + 0.0f; }

__device__ __forceinline__ float load_logit(const RouteArgs &a, int64_t t, int e)
{
    const float l = a.bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(a.logits)[t * a.ld + e]) << 16)
                           : static_cast<const float *>(a.logits)[t * a.ld + e];
    return finite_logit(l);
}

__device__ __forceinline__ float fast_exp(float v) { return __expf(v); }
__device__ __forceinline__ double fast_exp(double v) { return exp(v); }
__device__ __forceinline__ float fast_inverse(float v) { return __fdividef(1.0f, v); }
__device__ __forceinline__ double fast_inverse(double v) { return 1.0 / v; }

// Chosen experts of one token: lane j < top holds the j-th (-1: none).  Returns
// false (all lanes) where fp32 scores cannot decide.  lmax and sum receive what p
// needs: the largest logit and the sum of exponentials (softmax).
// Lane l holds experts [l V, l V + V): of equal keys the lowest lane's first one
// is the lowest expert.
template <typename T, int V>
__device__ __forceinline__ bool choose(const RouteArgs &a, const float (&l)[V], bool by_logit, int lane, int &mine, float &lmax, T &sum)
{
    using Key = decltype(key_of(T()));
    if (!a.sigmoid) {
        float mx = l[0];
#pragma unroll
        for (int i = 1; i < V; ++i) mx = fmaxf(mx, l[i]);
        lmax = value_of(warp_max(key_of(mx)));
        T s = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) s += l[i] == -INFINITY ? T(0) : fast_exp(static_cast<T>(l[i]) - static_cast<T>(lmax));
        sum = warp_sum(s);
    }
    const T inv = a.sigmoid ? T(0) : fast_inverse(sum);
    Key key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        T v = static_cast<T>(l[i]);
        if (!by_logit) {
            v = a.sigmoid ? fast_inverse(T(1) + fast_exp(-v)) : fast_exp(v - static_cast<T>(lmax)) * inv;
            if (a.bias && e < a.E) v += static_cast<T>(__ldg(a.bias + e));
        }
        key[i] = l[i] == -INFINITY ? Key(0) : key_of(v);
    }
    bool sure = true;
    if (a.groups > 1) {
        const int per = a.E / a.groups;
        const int span = per / V;                // lanes per group
        // A group of whole lanes, as many as a power of two: its two best by exchanges
        // inside the group.  gkey: what the lane's group counts (0: no expert left).
        const bool by_lanes = per % V == 0 && (span & (span - 1)) == 0;
        Key gkey = 0;
        float gsize = 0.0f;                      // the scores' magnitudes in gkey
        int group = lane;                        // whose worth gkey is
        if (by_lanes) {
            Key k1 = 0, k2 = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                k2 = max(k2, min(k1, key[i]));
                k1 = max(k1, key[i]);
            }
            for (int o = 1; o < span; o <<= 1) {
                const Key o1 = __shfl_xor_sync(0xFFFFFFFFu, k1, o), o2 = __shfl_xor_sync(0xFFFFFFFFu, k2, o);
                k2 = max(max(k2, o2), min(k1, o1));
                k1 = max(k1, o1);
            }
            if (k1) {
                const bool two = a.group_top > 1 && k2;
                gkey = two ? key_of(value_of(k1) + value_of(k2)) : k1;
                gsize = fabsf(static_cast<float>(value_of(k1))) + (two ? fabsf(static_cast<float>(value_of(k2))) : 0.0f);
            }
            group = lane / span;
        } else {
            for (int g = 0; g < a.groups; ++g) {
                T worth = 0;
                float size = 0.0f;
                bool some = false;
                int skip = -1;
                for (int n = 0; n < a.group_top; ++n) {
                    Key best = 0;
                    int at = 0x7FFFFFFF;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int e = lane * V + i;
                        if (e >= g * per && e < (g + 1) * per && e != skip && key[i] > best) { best = key[i]; at = e; }
                    }
                    const Key top = warp_max(best);
                    if (top == 0) break;
                    skip = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(best == top ? at : 0x7FFFFFFF)));
                    worth += value_of(top);
                    size += fabsf(static_cast<float>(value_of(top)));
                    some = true;
                }
                if (lane == g) {
                    gkey = some ? key_of(worth) : Key(0);
                    gsize = size;
                }
            }
        }
        uint32_t open = 0;                       // bit g: group g is kept
        T last = 0;
        for (int n = 0; n <= a.keep && n < a.groups; ++n) {
            const Key rest = (open >> group) & 1u ? Key(0) : gkey;
            const Key best = warp_max(rest);
            if (best == 0) break;
            const T v = value_of(best);
            if (n == a.keep) {
                // (any group may be the one whose error crosses the border: the largest counts)
                if (!by_logit) {
                    const float size = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(gsize)));
                    if (too_close(last, v, 2.0f * fmaxf(1.0f, size))) sure = false;
                }
                break;
            }
            const int who = __ffs(__ballot_sync(0xFFFFFFFFu, rest == best)) - 1;
            open |= 1u << (by_lanes ? who / span : who);
            last = v;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            if (e < a.E && !((open >> (by_lanes ? group : e / per)) & 1u)) key[i] = 0;
        }
    }
    mine = -1;
    T last = 0;
    for (int n = 0; n <= a.top; ++n) {
        Key best = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) best = max(best, key[i]);
        const Key top = warp_max(best);
        if (top == 0) break;
        if (!by_logit) {
            const T v = value_of(top);
            if (n > 0 && too_close(last, v, fmaxf(fabsf(static_cast<float>(last)), fabsf(static_cast<float>(v))))) sure = false;
            last = v;
        }
        if (n == a.top) break;
        const int who = __ffs(__ballot_sync(0xFFFFFFFFu, best == top)) - 1;
        int at = 0;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (key[i] == top) at = i;           // the first of them
        const int e = __shfl_sync(0xFFFFFFFFu, lane * V + at, who);
        if (lane == n) mine = e;
        if (lane == who) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == at) key[i] = 0;
        }
    }
    return sure;
}

// (registers for 12 CTAs per SM with 4 logits a lane: left to itself the compiler takes 32, for
// 16 CTAs; 8192 tokens, 8 of 128: 7.5 us against 8.1 us)
template <int V>
__global__ void __launch_bounds__(32 * RT_WARPS, V <= 4 ? 12 : V <= 8 ? 10 : 6) route_kernel(const RouteArgs a)
{
    sqd::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
    const int64_t t = static_cast<int64_t>(blockIdx.x) * RT_WARPS + (threadIdx.x >> 5);
    sqd::pdl_wait();
    if (t >= a.T) return;
    float l[V];
    if (a.vec) {
        // the lane's V logits by 16-byte loads (every row starts on one, and E = 32 V)
        uint32_t u[V];
        const int n = a.bf16 ? V / 8 : V / 4;
        const uint4 *row = static_cast<const uint4 *>(a.logits) + (t * a.ld + lane * V) / (a.bf16 ? 8 : 4);
#pragma unroll
        for (int i = 0; i < (V + 3) / 4; ++i)
            if (i < n) {
                const uint4 v = row[i];
                if (V >= 4) { u[(4 * i) % V] = v.x; u[(4 * i + 1) % V] = v.y; u[(4 * i + 2) % V] = v.z; u[(4 * i + 3) % V] = v.w; }
            }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t w = a.bf16 ? ((i & 1) ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16) : u[i];
            l[i] = finite_logit(__uint_as_float(w));
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = lane * V + i < a.E ? load_logit(a, t, lane * V + i) : -INFINITY;
    }
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
// index outside [0, E); offsets[E + 1].  One cluster of up to 8 CTAs: every warp
// owns a contiguous range of pairs and counts its experts; after sums over the
// warps, the CTAs (their totals read through distributed shared memory) and the
// experts, each gives out rows in order, 32 pairs at a time (lanes with the same
// expert rank themselves by lane).  No atomics decide an order.
// 32768 pairs of 64 experts: 31.5 us on one CTA, whose 32 warps share one SM's
// matching and shared-memory atomics.
constexpr int DP_WARPS = 32;
constexpr int DP_UNROLL = 8;      // ids in flight per lane
constexpr int DP_CTAS = 8;
constexpr int DP_PAIRS = 2048;    // pairs per CTA from which another CTA pays

__global__ void __launch_bounds__(32 * DP_WARPS) dispatch_kernel(const int32_t *__restrict__ ids, int64_t pairs, int E,
                                                                 int32_t *__restrict__ offsets, int32_t *__restrict__ pos)
{
    extern __shared__ int32_t cnt[];   // [DP_WARPS][E], then [E + 1] offsets, then the CTA's [E] totals
    int32_t *off = cnt + DP_WARPS * E, *tot = off + E + 1;
    sqd::pdl_launch_dependents();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int ctas = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);   // one cluster
    const int64_t per = ((pairs + DP_WARPS * ctas - 1) / (DP_WARPS * ctas) + 31) / 32 * 32;
    const int64_t lo = min(per * (rank * DP_WARPS + w), pairs), hi = min(lo + per, pairs);
    for (int i = threadIdx.x; i < DP_WARPS * E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    sqd::pdl_wait();
    int32_t *mine = cnt + w * E;
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * DP_UNROLL) {
        int e[DP_UNROLL];
#pragma unroll
        for (int u = 0; u < DP_UNROLL; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            e[u] = i < hi ? ids[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < DP_UNROLL; ++u)
            if (e[u] >= 0 && e[u] < E) atomicAdd(mine + e[u], 1);
    }
    __syncthreads();
    // counts -> first row of every (warp, expert), relative to the CTA's first of that expert
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int32_t s = 0;
#pragma unroll 8
        for (int v = 0; v < DP_WARPS; ++v) {
            const int32_t c = cnt[v * E + e];
            cnt[v * E + e] = s;
            s += c;
        }
        tot[e] = s;
    }
    if (ctas > 1) sqd::cluster_sync();   // every CTA's totals stand
    else __syncthreads();
    int32_t before[(MAX_EXPERTS + 32 * DP_WARPS - 1) / (32 * DP_WARPS)];   // of the CTAs before this one
#pragma unroll
    for (int q = 0; q < static_cast<int>(sizeof(before) / sizeof(int32_t)); ++q) {
        const int e = threadIdx.x + q * 32 * DP_WARPS;
        before[q] = 0;
        if (e >= E) continue;
        int32_t all = 0;
        for (int c = 0; c < ctas; ++c) {
            int32_t v;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(sqd::map_to_cta(sqd::smem_u32(tot + e), c)) : "memory");
            if (c < rank) before[q] += v;
            all += v;
        }
        off[e + 1] = all;
    }
    if (ctas > 1) sqd::cluster_sync();   // the totals are read: tot takes what comes before
    else __syncthreads();
#pragma unroll
    for (int q = 0; q < static_cast<int>(sizeof(before) / sizeof(int32_t)); ++q) {
        const int e = threadIdx.x + q * 32 * DP_WARPS;
        if (e < E) tot[e] = before[q];
    }
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
    if (rank == 0)
        for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = off[e];
    for (int e = lane; e < E; e += 32) mine[e] += off[e] + tot[e];
    __syncwarp();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * DP_UNROLL) {
        int e[DP_UNROLL];
#pragma unroll
        for (int u = 0; u < DP_UNROLL; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            e[u] = i < hi ? ids[i] : -1;
            if (e[u] >= E) e[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < DP_UNROLL; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, e[u]);
            const int rank = __popc(same & ((1u << lane) - 1u));
            int32_t r = -1;
            if (e[u] >= 0) r = mine[e[u]] + rank;
            __syncwarp();
            if (e[u] >= 0 && rank == 0) mine[e[u]] += __popc(same);
            __syncwarp();
            if (i < hi) pos[i] = r;
        }
    }
}

// ---------------------------------------------------------------- dispatch and quantizer for a few tokens
// dispatch_kernel and the block quantizer's scattered form in one launch, for up to
// 256 pairs: every CTA counts all pairs itself (a histogram and a scan over the
// experts), each warp takes 256 channels of one copy of one token, and CTA (0, 0)
// writes offsets and pos.  The experts of one token of 4096 channels, 8 of 64: 35.5 us
// a call against 39.6 us with the two launches.
constexpr int DQ_PAIRS = 256;

__global__ void __launch_bounds__(sqb::QB_THREADS) dispatch_quant_kernel(const int32_t *__restrict__ ids, int T, int top, int E,
                                                                         int32_t *__restrict__ offsets, int32_t *__restrict__ pos,
                                                                         const uint16_t *__restrict__ X, int K, int64_t ldx,
                                                                         int k_pad, int s_ld, uint8_t *__restrict__ X_8,
                                                                         float *__restrict__ s_x)
{
    __shared__ int32_t id[DQ_PAIRS];
    __shared__ int32_t off[MAX_EXPERTS + 1];   // counts of expert e at e + 1, then their running sum
    sqd::pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31;
    const int pairs = T * top;
    for (int e = tid; e <= E; e += sqb::QB_THREADS) off[e] = 0;
    __syncthreads();
    sqd::pdl_wait();
    if (tid < pairs) {
        int e = ids[tid];
        if (e < 0 || e >= E) e = -1;
        id[tid] = e;
        if (e >= 0) atomicAdd(&off[e + 1], 1);
    }
    __syncthreads();
    if (tid < 32) {
        int32_t base = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            int32_t v = e0 + lane < E ? off[e0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o) v += u;
            }
            if (e0 + lane < E) off[e0 + lane + 1] = base + v;
            base += __shfl_sync(0xFFFFFFFFu, v, 31);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        for (int e = tid; e <= E; e += sqb::QB_THREADS) offsets[e] = off[e];
        if (tid < pairs) {
            int32_t r = -1;
            if (id[tid] >= 0) {
                r = off[id[tid]];
                for (int j = 0; j < tid; ++j) r += id[j] == id[tid];
            }
            pos[tid] = r;
        }
    }
    const int segs = (s_ld * sqb::BLK + 255) / 256;
    const int w = blockIdx.x * (sqb::QB_THREADS / 32) + (tid >> 5);
    if (w >= T * segs) return;
    const int t = w / segs, pair = t * top + static_cast<int>(blockIdx.y);
    const int e = id[pair];
    if (e < 0) return;
    int64_t d = off[e];
    for (int j0 = 0; j0 < pair; j0 += 32) d += __popc(__ballot_sync(0xFFFFFFFFu, j0 + lane < pair && id[j0 + lane] == e));
    const int c = (w - t * segs) * 32 + lane;
    const uint4 v = c < (K >> 3) ? sqd::ld_nc_v4(X + t * ldx + 8 * c) : make_uint4(0, 0, 0, 0);
    uint32_t m = sqb::absmax8(v);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const sqb::BlockScale b = sqb::block_scale(__uint_as_float(m << 16));
    if (8 * c < k_pad) *reinterpret_cast<uint2 *>(X_8 + d * k_pad + 8 * c) = sqb::block_codes(v, b);
    if ((lane & 15) == 0 && (c >> 4) < s_ld) s_x[d * s_ld + (c >> 4)] = b.s;
}

// ---------------------------------------------------------------- combine
// Y[t] = sum_j weights[t, j] Z[pos[t, j]] over the choices that have a row, in
// the order of j, fp32, rounded once.  One thread per 8 columns; the rows of Z
// that have no choice are never read.  Memory-bound: top + 1 rows of 2 N bytes,
// 4096 tokens of 4096 columns: 8 choices 53 us (46 us at the copy rate), 2 choices
// 24 us (15 us; with code for 8 in flight 33 us, and 43 us when the token's index
// was a 64-bit quotient).
constexpr int CB_THREADS = 256;

template <int FLIGHT>
__global__ void __launch_bounds__(CB_THREADS) combine_kernel(const uint16_t *__restrict__ Z, int64_t rows_z, int64_t ldz,
                                                             const int32_t *__restrict__ pos, const float *__restrict__ weights,
                                                             int64_t T, int top, int N, uint16_t *__restrict__ Y, int64_t ldy)
{
    sqd::pdl_launch_dependents();
    sqd::pdl_wait();
    const int per = N >> 3;
    const int64_t total = T * per;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = total <= 0xFFFFFFFFll ? static_cast<uint32_t>(i) / static_cast<uint32_t>(per) : i / per;
        const int c = static_cast<int>(i - t * per) * 8;
        float acc[8] = {};
        for (int j0 = 0; j0 < top; j0 += FLIGHT) {
            int32_t r[FLIGHT];
            float w[FLIGHT];
            uint4 v[FLIGHT];
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j) {
                r[j] = j0 + j < top ? pos[t * top + j0 + j] : -1;
                w[j] = j0 + j < top ? weights[t * top + j0 + j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j)
                v[j] = r[j] >= 0 && r[j] < rows_z ? *reinterpret_cast<const uint4 *>(Z + r[j] * ldz + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j) {
                if (r[j] < 0 || r[j] >= rows_z) continue;
                const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    acc[2 * q] = fmaf(w[j], __uint_as_float(u[q] << 16), acc[2 * q]);
                    acc[2 * q + 1] = fmaf(w[j], __uint_as_float(u[q] & 0xFFFF0000u), acc[2 * q + 1]);
                }
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
