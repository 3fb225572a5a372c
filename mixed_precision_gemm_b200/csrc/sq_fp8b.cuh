// Block-scaled FP8: E4M3 codes with one fp32 scale for each 128 channels of a
// token (X) or each 128 x 128 block of the weights (W).
//
//   s = fl(a / 448), a the block's largest magnitude; s == 0 (a == 0, or fp32 values
//   so small that the quotient rounds to 0): codes 0
//   e(x) = the E4M3 code nearest to fl(x / s), ties to even
//   Y[m,n] = sum_b sx[m,b] sw[n/128,b] sum_{k in block b} e(X)[m,k] e(W)[n,k]
//
// Storage: codes [rows, k_pad] bytes, k_pad = roundup(K, 128), zero past K;
// scales [rows or row blocks, s_ld] floats, s_ld = roundup(K, 512) / 128, zero
// past the last block (so a row's scales can be read four at a time).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sq_device.cuh"
#include "sq_rowquant.cuh"

namespace sqb {

constexpr int BLK = 128;        // channels (and weight rows) per scale
constexpr float kTop = 448.0f;  // largest E4M3 magnitude

// ---------------------------------------------------------------- quantizers
// Scale of a block from the bits of its largest bf16 magnitude, and the
// constants of the quotient (sq_rowquant.cuh: correctly rounded x / s).
struct BlockScale {
    float s;
    bool zero, up;
    sqq::RowScale rs;
};

__device__ __forceinline__ BlockScale block_scale(float amax)
{
    BlockScale b;
    b.s = sqq::row_scale(amax, kTop, 1.0f / kTop);   // (0 for 0)
    b.zero = b.s == 0.0f;   // (a bf16 magnitude over 448 is an fp32 number; one of h need not be)
    b.up = !b.zero && b.s < sqq::kTinyScale;
    const float s1 = b.up ? b.s * sqq::kUpScale : b.s;
    const float inv = b.zero ? 0.0f : __frcp_rn(s1);
    b.rs.inv2 = sqq::f2_pack(__float_as_uint(inv), __float_as_uint(inv));
    b.rs.negs2 = sqq::f2_pack(__float_as_uint(-s1), __float_as_uint(-s1));
    b.rs.magic2 = 0;
    b.rs.up2 = sqq::f2_pack(__float_as_uint(sqq::kUpScale), __float_as_uint(sqq::kUpScale));
    return b;
}

__device__ __forceinline__ uint2 block_codes(const uint4 &v, const BlockScale &b)
{
    uint2 c = make_uint2(0u, 0u);
    if (b.zero) return c;
    if (!b.up) sqq::quant8_fp8_pairs<false>(v, b.rs, c.x, c.y);
    else sqq::quant8_fp8_pairs<true>(v, b.rs, c.x, c.y);
    return c;
}

// Largest magnitude of 8 bf16 values, as bf16 bits.
__device__ __forceinline__ uint32_t absmax8(const uint4 &v)
{
    const uint32_t m = sqq::maxabs_bf16x2(sqq::maxabs_bf16x2(v.x, v.y), sqq::maxabs_bf16x2(v.z, v.w)) & 0x7FFF7FFFu;
    return max(m & 0xFFFFu, m >> 16);
}

constexpr int QB_THREADS = 256;

// Codes and scales of the rows of X.  One warp takes 256 CHUNKS channels of a row:
// lane l holds chunks l, l + 32, ... of 8 channels (16 bytes), so 16 lanes
// share a block of 128 and its maximum takes four shuffles.
// With pos (top > 0) row t of X goes to the `top` rows pos[t * top + j] of the
// outputs (entries outside [0, rows_out) are skipped): one read of a token for all
// of its experts' copies; a token without any is not read.  With few tokens
// (gridDim.y = top) a warp writes one copy only.
// Memory-bound: 2 K bytes read and (K + 4 K / 128) written per output row.
template <int CHUNKS>
__global__ void __launch_bounds__(QB_THREADS) quant_kernel(const uint16_t *__restrict__ X, int64_t rows, int K, int64_t ldx,
                                                           int k_pad, int s_ld, const int32_t *__restrict__ pos, int top,
                                                           int64_t rows_out, uint8_t *__restrict__ X_8,
                                                           float *__restrict__ s_x)
{
    constexpr int SEG = 32 * CHUNKS * 8;
    const int lane = threadIdx.x & 31;
    const int segs = (s_ld * BLK + SEG - 1) / SEG;
    const int64_t tasks = rows * segs;
    const int64_t wpg = static_cast<int64_t>(gridDim.x) * (QB_THREADS / 32);
    const int j_lo = gridDim.y > 1 ? blockIdx.y : 0, j_hi = gridDim.y > 1 ? j_lo + 1 : max(top, 1);
    sqd::pdl_wait();
    sqd::pdl_launch_dependents();   // (here: whoever starts now finds what came before this kernel complete)
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * (QB_THREADS / 32) + (threadIdx.x >> 5); w < tasks; w += wpg) {
        const int64_t r = tasks <= 0xFFFFFFFFll ? static_cast<uint32_t>(w) / static_cast<uint32_t>(segs) : w / segs;
        const int c0 = static_cast<int>(w - r * segs) * (SEG / 8) + lane;
        int32_t dst = -1;                       // lane j: the row's j-th copy
        if (top > 0) {
            if (lane >= j_lo && lane < j_hi) dst = pos[r * top + lane];
            if (dst >= rows_out) dst = -1;
            if (!__any_sync(0xFFFFFFFFu, dst >= 0)) continue;
        }
        const uint16_t *row = X + r * ldx;
        uint4 v[CHUNKS];
        uint2 q[CHUNKS];
        float sc[CHUNKS];
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int c = c0 + 32 * i;
            v[i] = c < (K >> 3) ? sqd::ld_nc_v4(row + 8 * c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            uint32_t m = absmax8(v[i]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const BlockScale b = block_scale(__uint_as_float(m << 16));
            q[i] = block_codes(v[i], b);
            sc[i] = b.s;
        }
        for (int j = j_lo; j < j_hi; ++j) {
            const int64_t d = top > 0 ? __shfl_sync(0xFFFFFFFFu, dst, j) : r;
            if (d < 0) continue;
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                const int c = c0 + 32 * i;
                if (8 * c < k_pad) *reinterpret_cast<uint2 *>(X_8 + d * k_pad + 8 * c) = q[i];
                if ((lane & 15) == 0 && (c >> 4) < s_ld) s_x[d * s_ld + (c >> 4)] = sc[i];
            }
        }
    }
}

// Codes and scales of weight blocks: CTA (kb, nb, g) takes the 128 x 128 block
// (nb, kb) of matrix g.  Thread t holds chunk t % 16 of rows t / 16, + 16, ...
// The blocks past the last one of a scale row (kb up to s_ld) only write their 0.
__global__ void __launch_bounds__(256) weight_blocks_kernel(const uint16_t *__restrict__ W, int N, int K, int64_t ldw,
                                                            int64_t stride_g, int k_pad, int s_ld,
                                                            uint8_t *__restrict__ W_8, float *__restrict__ s_w)
{
    sqd::pdl_launch_dependents();
    __shared__ uint32_t red[8];
    const int kb = blockIdx.x, nb = blockIdx.y;
    const int64_t g = blockIdx.z;
    const int c = kb * 16 + (threadIdx.x & 15);
    const int r0 = nb * BLK + (threadIdx.x >> 4);
    sqd::pdl_wait();
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        v[i] = (r < N && c < (K >> 3)) ? sqd::ld_nc_v4(W + g * stride_g + r * ldw + 8 * c) : make_uint4(0, 0, 0, 0);
        m = max(m, absmax8(v[i]));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, red[i]);
    const BlockScale b = block_scale(__uint_as_float(m << 16));
    if (threadIdx.x == 0) s_w[(g * gridDim.y + nb) * s_ld + kb] = b.s;
    if (8 * c >= k_pad) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        if (r < N) *reinterpret_cast<uint2 *>(W_8 + (g * N + r) * k_pad + 8 * c) = block_codes(v[i], b);
    }
}

// ---------------------------------------------------------------- products
// One product, or one per expert: rows [offsets[g], offsets[g + 1]) of X take
// matrix g.  Without offsets, one matrix takes rows [0, M).
struct ProductArgs {
    const uint8_t *X_8;
    const float *s_x;
    const uint8_t *W_8;      // [G, (2,) N, k_pad]
    const float *s_w;        // [G, (2,) nb, s_ld]
    const int32_t *offsets;  // [G + 1], or NULL
    int64_t M;               // rows of X_8 (capacity where there are offsets)
    int G, N, kb, k_pad, s_ld, nb;
    uint16_t *Y;             // bf16 [M, ldy]
    int64_t ldy;
    uint8_t *H_8;            // SwiGLU form: codes [M, h_pad] and scales [M, h_ld]
    float *s_h;
    int h_pad, h_ld;
    // The kernel right before this one in the stream writes neither the weights nor
    // offsets, and lets its successors start only once all before it has ended.
    bool settled;
};

// Rows of expert g, clamped to the buffers whatever the offsets hold.
__device__ __forceinline__ void expert_rows(const ProductArgs &a, int g, int64_t &lo, int64_t &hi)
{
    if (!a.offsets) {
        lo = 0;
        hi = a.M;
        return;
    }
    lo = min(max(static_cast<int64_t>(a.offsets[g]), int64_t(0)), a.M);
    hi = min(max(static_cast<int64_t>(a.offsets[g + 1]), lo), a.M);
}

// silu(g) u of two columns with the hardware's exponential and reciprocal: one MUFU
// each where expf and an exact quotient cost some 30 instructions, the rest packed.
// Off by about 2^-21 of the value near g = 0; for negative g the rounding of the
// exponential's argument adds 0.4 |g| 2^-23 (2^-20 at -20, 2^-18 at -87), far below
// what the products' errors, 2^-12 of their terms' magnitudes, do to it.  From
// e^-g = 2^126 on (g = -87.3) the value is 0, of a silu below 2^-119.
__device__ __forceinline__ float2 silu_mul2(float2 g, float2 u)
{
    const float2 t = __fmul2_rn(g, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    e = __fadd2_rn(e, make_float2(1.0f, 1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    return __fmul2_rn(__fmul2_rn(g, r), u);
}

// A block's scale and what its codes need: the scale's inverse and negative, of a
// scale brought up by 2^64 if it is tiny (the values have to be, too).  A block of
// scale 0 takes its values times 0, and zeros of either sign to code 0.
struct CodeScale {
    float s, inv, neg, up;
};

__device__ __forceinline__ CodeScale code_scale(float amax)
{
    const BlockScale b = block_scale(amax);
    CodeScale c;
    uint32_t inv, neg, hi;
    sqq::f2_unpack(b.rs.inv2, inv, hi);
    sqq::f2_unpack(b.rs.negs2, neg, hi);
    c.s = b.s;
    c.inv = b.zero ? 1.0f : __uint_as_float(inv);
    c.neg = b.zero ? -1.0f : __uint_as_float(neg);
    c.up = b.zero ? 0.0f : b.up ? sqq::kUpScale : 1.0f;
    return c;
}

// E4M3 codes of two (brought up) fp32 values, in the low 16 bits: the rounded
// quotients as in sq_rowquant.cuh.
__device__ __forceinline__ uint32_t codes2(float2 v, float2 inv, float2 neg)
{
    const float2 q0 = __fmul2_rn(v, inv);
    const float2 q1 = __ffma2_rn(__ffma2_rn(q0, neg, v), inv, q0);
    return __nv_cvt_float2_to_fp8x2(q1, __NV_SATFINITE, __NV_E4M3);
}

}  // namespace sqb
