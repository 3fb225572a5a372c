// Block-scaled FP8 products for few rows per weight matrix: swapped operands, K
// split over a cluster.  Same computation as sq_fp8b_pair.cuh.
//
// The product is a stream over the weights.  A tile is 128 weight rows (one row
// of scale blocks; SwiGLU: 128 gate rows and the same 128 up rows) by MP rows of
// X, as D^T = W X^T: the weight rows are the MMA's M side (TMEM lanes) and the MP
// rows of X its N side, so that few rows cost little.  Each 128-channel block of
// D^T goes to a small ring of TMEM buffers; four epilogue warps (a thread per
// weight row) add it, times sx[m,b] sw[b], to MP sums in registers.  sx sw of four
// blocks at a time is a table in shared memory, read as broadcasts.
//
// The blocks of a tile are divided over the S <= 8 CTAs of a cluster, so that few
// tiles still occupy every SM.  CTA r of the cluster owns the tile's rows of X
// [r TP, (r + 1) TP), TP = ceil(MP / S): every CTA sends the owner its sums through
// distributed shared memory (the operand ring, free by then), and the owner adds
// them in rank order and stores; in the SwiGLU form it has the 128 columns of h
// that share a scale, and writes their codes.
//
// Memory-bound on the weights; two CTAs fit on an SM (one where the tile is
// large), so that one loads while the other starts or finishes.
//
// Roles (6 warps): 0 loads (TMA), 1 issues the MMAs, 2..5 sums.
#pragma once

#include "sq_fp8b.cuh"

namespace sqb {

constexpr int SB_THREADS = 192;
constexpr int SB_MAX_SPLITS = 8;

enum : unsigned { SITE_SB_LOAD = 0x701, SITE_SB_MMA = 0x702, SITE_SB_EPI = 0x703 };

template <int MP_, bool SWIGLU_, int NST_, int PER_SM_>
struct CfgSkinnyB {
    static constexpr int MP = MP_, NST = NST_, PER_SM = PER_SM_;
    static constexpr bool SWIGLU = SWIGLU_;
    static constexpr int MATS = SWIGLU ? 2 : 1;
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int STAGE = MATS * W_BYTES + MP * 128;
    static constexpr int COLS = MATS * MP;                       // TMEM columns per block
    static constexpr int NB = 256 / COLS < 4 ? 256 / COLS : 4;   // TMEM buffers
    static constexpr int TMEM = NB * COLS <= 32 ? 32 : NB * COLS <= 64 ? 64 : NB * COLS <= 128 ? 128 : 256;
    static constexpr int OFF_TAB = NST * STAGE;                  // [2][4][MATS][MP] products of scales
    static constexpr int OFF_MAX = OFF_TAB + 2 * 4 * MATS * MP * 4;   // [4 warps][MP] maxima
    static constexpr int OFF_BAR = OFF_MAX + (SWIGLU ? 4 * MP * 4 : 0);
    static constexpr int NBAR = 2 * NST + 2 * NB + 1;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;          // TMEM address, abort flag, tile
    static constexpr int SMEM = OFF_MISC + 32 + 1024;
    static_assert(STAGE % 1024 == 0, "swizzled tiles");
    static_assert(MATS * (MP + SB_MAX_SPLITS - 1) * 512 <= NST * STAGE, "the exchanged sums fit in the ring");
    static_assert(SMEM * PER_SM <= 232448 && TMEM * PER_SM <= 512, "an SM's share");
};

struct SkinnyBArgs {
    ProductArgs p;
    int splits;
};

// Tile index -> expert, its first row of X in the tile and its end, weight tile.
// Tiles of an expert: its row chunks fastest, so that those that share weight
// rows run together.  Called by one whole warp; false behind the last tile.
__device__ __forceinline__ bool skinny_tile(const ProductArgs &a, int mp, int t, int lane, int &g, int &m0, int &m_end, int &tn)
{
    int base = 0;
    for (int g0 = 0; g0 < a.G; g0 += 32) {
        int64_t lo = 0, hi = 0;
        if (g0 + lane < a.G) expert_rows(a, g0 + lane, lo, hi);
        const int chunks = static_cast<int>((hi - lo + mp - 1) / mp);
        int sum = chunks * a.nb;
        const int mine = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += u;
        }
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, t < base + sum);
        if (who) {
            const int l = __ffs(who) - 1;
            const int first = __shfl_sync(0xFFFFFFFFu, base + sum - mine, l);
            const int c = __shfl_sync(0xFFFFFFFFu, chunks, l);
            const int row = static_cast<int>(__shfl_sync(0xFFFFFFFFu, static_cast<int>(lo), l));
            m_end = static_cast<int>(__shfl_sync(0xFFFFFFFFu, static_cast<int>(hi), l));
            g = g0 + l;
            tn = (t - first) / c;
            m0 = row + (t - first) % c * mp;
            return true;
        }
        base += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    return false;
}

template <class C>
__global__ void __launch_bounds__(SB_THREADS, C::PER_SM)
product_skinny_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const SkinnyBArgs args)
{
    constexpr int MP = C::MP, NST = C::NST, NB = C::NB, MATS = C::MATS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = sqd::smem_u32(smem);
    const ProductArgs &p = args.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = args.splits;
    const int rank = static_cast<int>(sqd::cluster_ctarank());
    sqd::pdl_launch_dependents();

    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (NST + s); };
    auto bfull = [&](int j) { return bar0 + 8u * (2 * NST + j); };
    auto bempty = [&](int j) { return bar0 + 8u * (2 * NST + NB + j); };
    const uint32_t drain = bar0 + 8u * (2 * NST + 2 * NB);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + C::OFF_MISC + 4);
    int *where = reinterpret_cast<int *>(smem + C::OFF_MISC + 8);   // expert, first row, end, weight tile, any
    auto stage = [&](int s) { return sbase + s * C::STAGE; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            sqd::mbar_init(full(s), 1);
            sqd::mbar_init(empty(s), 1);
        }
        for (int j = 0; j < NB; ++j) {
            sqd::mbar_init(bfull(j), 1);
            sqd::mbar_init(bempty(j), 4);
        }
        sqd::mbar_init(drain, 1);
        *abort_flag = 0u;
        sqd::fence_barrier_init();
        sqd::fence_proxy_async_smem();
        sqd::prefetch_tensormap(&tm_x);
        sqd::prefetch_tensormap(&tm_w);
    }
    if (warp == 1) {
        sqd::tmem_alloc(sqd::smem_u32(tmem_slot), C::TMEM);
        sqd::tmem_relinquish();
    }
    sqd::pdl_wait();  // operands, offsets and outputs may belong to the previous kernel
    if (warp == 0) {
        int g = 0, m0 = 0, m_end = 0, tn = 0;
        const bool any = skinny_tile(p, MP, static_cast<int>(blockIdx.x) / S, lane, g, m0, m_end, tn);
        if (lane == 0) {
            where[0] = g;
            where[1] = m0;
            where[2] = m_end;
            where[3] = tn;
            where[4] = any;
        }
    }
    sqd::tc_fence_before();
    __syncthreads();
    sqd::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int g = where[0], m0 = where[1], m_end = where[2], tn = where[3];
    const bool any = where[4] != 0;   // the same in every CTA of the cluster
    if (!any) {
        if (warp == 1) sqd::tmem_dealloc(tmem, C::TMEM);
        return;
    }
    const int b_lo = static_cast<int>(static_cast<int64_t>(p.kb) * rank / S);
    const int nblk = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / S) - b_lo;

    float2 acc[MATS][MP / 2];
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int s = 0, last = -1;
            uint32_t ph = 0, last_ph = 0;
            bool ok = true;
            for (int i = 0; i < nblk; ++i) {
                if (!sqd::mbar_wait(empty(s), ph ^ 1u, abort_flag, SITE_SB_LOAD)) { ok = false; break; }
                sqd::mbar_arrive_expect_tx(full(s), C::STAGE);
                const int x = (b_lo + i) * BLK;
#pragma unroll
                for (int mat = 0; mat < MATS; ++mat)
                    sqd::tma_load_2d(stage(s) + mat * C::W_BYTES, &tm_w, full(s), x, (g * MATS + mat) * p.N + tn * 128);
                sqd::tma_load_2d(stage(s) + MATS * C::W_BYTES, &tm_x, full(s), x, m0);
                last = s;
                last_ph = ph;
                if (++s == NST) { s = 0; ph ^= 1u; }
            }
            if (!ok && last >= 0) sqd::mbar_drain(full(last), last_ph);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        if (lane == 0) {
            constexpr uint32_t idesc = sqd::make_idesc_e4m3(128, MP);
            int s = 0, j = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true;
            for (int i = 0; i < nblk; ++i) {
                const uint64_t ad = sqd::make_sw128_desc(stage(s));
                const uint64_t bd = sqd::make_sw128_desc(stage(s) + MATS * C::W_BYTES);
                if (!sqd::mbar_wait(full(s), ph, abort_flag, SITE_SB_MMA) ||
                    !sqd::mbar_wait(bempty(j), bph ^ 1u, abort_flag, SITE_SB_MMA)) { ok = false; break; }
                sqd::tc_fence_after();
#pragma unroll
                for (int mat = 0; mat < MATS; ++mat)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sqd::mma_f8(tmem + j * C::COLS + mat * MP, ad + mat * (C::W_BYTES >> 4) + 2 * k, bd + 2 * k, idesc, k ? 1u : 0u);
                sqd::mma_commit(bfull(j));
                sqd::mma_commit(empty(s));
                if (++s == NST) { s = 0; ph ^= 1u; }
                if (++j == NB) { j = 0; bph ^= 1u; }
            }
            if (!ok) {
                sqd::mma_commit(drain);
                sqd::mbar_drain(drain, 0);
            }
        }
    } else {
        // ------------------------------------------------------------ sums
        // (a wait that gave up does not leave the loop, so that all four warps keep
        // meeting at the table's barrier; the tile is not stored then)
        const int et = threadIdx.x - 64;
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll
        for (int mat = 0; mat < MATS; ++mat)
#pragma unroll
            for (int c = 0; c < MP / 2; ++c) acc[mat][c] = make_float2(0.0f, 0.0f);
        float *tab = reinterpret_cast<float *>(smem + C::OFF_TAB);
        const bool row_ok = et < MP && m0 + et < m_end;
        const float4 *sx_p = reinterpret_cast<const float4 *>(p.s_x + static_cast<int64_t>(row_ok ? m0 + et : 0) * p.s_ld);
        const float4 *sw_p = reinterpret_cast<const float4 *>(p.s_w + (static_cast<int64_t>(g) * MATS * p.nb + tn) * p.s_ld);
        const int sw_up = p.nb * p.s_ld / 4;    // the up matrix's scales behind the gate's
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        float4 sx4 = z, sw4[MATS];
        auto fetch = [&](int q) {
            sx4 = row_ok ? __ldg(sx_p + q) : z;
#pragma unroll
            for (int mat = 0; mat < MATS; ++mat) sw4[mat] = __ldg(sw_p + mat * sw_up + q);
        };
        fetch(b_lo >> 2);
        int j = 0;
        uint32_t bph = 0;
        for (int i = 0; i < nblk; ++i) {
            const int b = b_lo + i, q = b >> 2;
            float *tq = tab + (q & 1) * (4 * MATS * MP);
            if (i == 0 || (b & 3) == 0) {
                if (et < MP) {
#pragma unroll
                    for (int mat = 0; mat < MATS; ++mat) {
                        tq[(0 * MATS + mat) * MP + et] = sx4.x * sw4[mat].x;
                        tq[(1 * MATS + mat) * MP + et] = sx4.y * sw4[mat].y;
                        tq[(2 * MATS + mat) * MP + et] = sx4.z * sw4[mat].z;
                        tq[(3 * MATS + mat) * MP + et] = sx4.w * sw4[mat].w;
                    }
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (((q + 1) << 2) < b_lo + nblk) fetch(q + 1);
            }
            sqd::mbar_wait(bfull(j), bph, abort_flag, SITE_SB_EPI);
            sqd::tc_fence_after();
            const float4 *tb = reinterpret_cast<const float4 *>(tq + (b & 3) * MATS * MP);
#pragma unroll
            for (int ch = 0; ch < C::COLS / 16; ++ch) {
                uint32_t v[16];
                sqd::tmem_ld_32x32b_x16(tl + j * C::COLS + 16 * ch, v);
                sqd::tmem_wait_ld_dep1(v);
                if (ch + 1 == C::COLS / 16) {
                    sqd::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) sqd::mbar_arrive(bempty(j));
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float4 s = tb[4 * ch + c];
                    float2 &a0 = acc[ch * 16 / MP][(ch * 16 % MP) / 2 + 2 * c], &a1 = acc[ch * 16 / MP][(ch * 16 % MP) / 2 + 2 * c + 1];
                    a0 = __ffma2_rn(make_float2(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1])), make_float2(s.x, s.y), a0);
                    a1 = __ffma2_rn(make_float2(__uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3])), make_float2(s.z, s.w), a1);
                }
            }
            if (++j == NB) { j = 0; bph ^= 1u; }
        }
    }

    // ---------------------------------------------------------------- exchange and store
    __syncwarp();
    sqd::fence_proxy_async_smem();   // the ring, filled by TMA and read by the MMAs, is written by threads below
    sqd::tc_fence_before();
    if (S > 1) sqd::cluster_sync();  // every MMA of the cluster is complete
    else __syncthreads();
    const int TP = (MP + S - 1) / S;
    const int et = static_cast<int>(threadIdx.x) - 64;
    if (warp >= 2) {
        // sums of row of X c to its owner: [mat][source][row of X][weight row]
        const int wr = (warp & 3) * 32 + lane;   // the thread's TMEM lane
        int owner = 0, cl = 0;
#pragma unroll
        for (int c = 0; c < MP; ++c) {
            const uint32_t off = static_cast<uint32_t>(((rank * TP + cl) * 128 + wr) * 4);
            const uint32_t dst = sqd::map_to_cta(sbase + off, static_cast<uint32_t>(owner));
#pragma unroll
            for (int mat = 0; mat < MATS; ++mat)
                sqd::st_cluster_f32(dst + static_cast<uint32_t>(mat * S * TP * 512), (c & 1) ? acc[mat][c / 2].y : acc[mat][c / 2].x);
            if (++cl == TP) { cl = 0; ++owner; }
        }
    }
    if (S > 1) sqd::cluster_sync();  // all sums delivered
    else __syncthreads();
    if (warp >= 2 && !*abort_flag) {
        float *red = reinterpret_cast<float *>(smem);
        const int n = tn * 128 + et;
        const int rows = min(min(TP, MP - rank * TP), m_end - m0 - rank * TP);   // owned rows that exist
        const int64_t mr = m0 + rank * TP;
        if constexpr (!C::SWIGLU) {
            for (int cl = 0; cl < rows; ++cl) {
                float s = 0.0f;
                for (int src = 0; src < S; ++src) s += red[(src * TP + cl) * 128 + et];
                if (n < p.N) p.Y[(mr + cl) * p.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
            }
        } else {
            float *wmax = reinterpret_cast<float *>(smem + C::OFF_MAX);
            for (int cl = 0; cl < rows; ++cl) {
                float gt = 0.0f, up = 0.0f;
                for (int src = 0; src < S; ++src) {
                    gt += red[(src * TP + cl) * 128 + et];
                    up += red[((S + src) * TP + cl) * 128 + et];
                }
                const float h = n < p.N ? silu_mul(gt, up) : 0.0f;
                red[cl * 128 + et] = h;
                const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(h)));
                if (lane == 0) wmax[(warp - 2) * MP + cl] = __uint_as_float(m);
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            // codes of four columns per thread: 32 threads a row, four rows at a time
            for (int cl = et >> 5; cl < rows; cl += 4) {
                const float mx = fmaxf(fmaxf(wmax[cl], wmax[MP + cl]), fmaxf(wmax[2 * MP + cl], wmax[3 * MP + cl]));
                const BlockScale bs = block_scale(mx);
                const float4 h = reinterpret_cast<const float4 *>(red + cl * 128)[lane];
                *reinterpret_cast<uint32_t *>(p.H_8 + (mr + cl) * p.h_pad + tn * 128 + 4 * lane) =
                    codes2(h.x, h.y, bs) | (codes2(h.z, h.w, bs) << 16);
                if (lane == 0) p.s_h[(mr + cl) * p.h_ld + tn] = bs.s;
                if (tn == p.nb - 1 && p.nb + lane < p.h_ld) p.s_h[(mr + cl) * p.h_ld + p.nb + lane] = 0.0f;
            }
        }
    }
    if (warp == 1) {
        sqd::tc_fence_after();
        sqd::tmem_dealloc(tmem, C::TMEM);
    }
}

}  // namespace sqb
