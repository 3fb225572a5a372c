// Block-scaled FP8 products for few rows per weight matrix: swapped operands, K
// split over a cluster.  Same computation as sq_fp8b_pair.cuh.
//
// The product is a stream over the weights.  A tile is 128 weight rows (one row
// of scale blocks; SwiGLU: 128 gate rows and the same 128 up rows) by MP rows of
// X, as D^T = W X^T: the weight rows are the MMA's M side (TMEM lanes) and the MP
// rows of X its N side, so that few rows cost little.  Each 128-channel block of
// D^T goes to the TMEM buffer of its ring stage; four epilogue warps (a thread per
// weight row) add it, times sx[m,b] sw[b], to MP sums in registers and give the
// stage, operands and buffer, back to the loads.  So the issuing thread has one
// wait and one commit per block: with a wait and a commit of its own for the
// buffers a block took it some 980 cycles, of which the MMAs are 512.  sx sw of
// four blocks at a time is a table in shared memory, read as broadcasts.
//
// With enough tiles for every SM the kernel is persistent (S = 1): each CTA takes
// every gridDim.x-th tile, its loads running ahead into the next tile while the
// sums of the last one are stored.  With fewer, the blocks of a tile are divided
// over the S <= 8 CTAs of a cluster (one tile per cluster).  The rows of X are then
// dealt out to the CTAs in fours: every CTA sends each row's owner its sums through
// distributed shared memory (the operand ring, free by then), and the owner adds
// them in rank order and stores.
// SwiGLU: whoever stores a row of X has the 128 columns of h that share a scale, and
// writes their codes.
//
// Memory-bound on the weights; two CTAs fit on an SM (one where the tile is large or
// the experts are many, CfgSkinnyB::per_sm), so that one loads while the other starts
// or finishes.
//
// Roles (6 warps): 0 loads (TMA), 1 issues the MMAs, 2..5 sums and stores.
#pragma once

#include "sq_fp8b.cuh"

namespace sqb {

constexpr int SB_THREADS = 192;
constexpr int SB_MAX_SPLITS = 8;
constexpr int SB_SM_BYTES = 233472;   // shared memory of an SM, 1 KB of it taken for each CTA

enum : unsigned { SITE_SB_LOAD = 0x701, SITE_SB_MMA = 0x702, SITE_SB_EPI = 0x703 };

template <int MP_, bool SWIGLU_, int NST_, int PER_SM_>
struct CfgSkinnyB {
    static constexpr int MP = MP_, NST = NST_, PER_SM = PER_SM_;
    static constexpr bool SWIGLU = SWIGLU_;
    static constexpr int MATS = SWIGLU ? 2 : 1;
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int STAGE = MATS * W_BYTES + MP * 128;
    static constexpr int COLS = MATS * MP;                       // TMEM columns per block
    static constexpr int TMEM = NST * COLS <= 32 ? 32 : NST * COLS <= 64 ? 64 : NST * COLS <= 128 ? 128 : NST * COLS <= 256 ? 256 : 512;
    static constexpr int OFF_TAB = NST * STAGE;                  // [2][4][MATS][MP] products of scales
    static constexpr int OFF_MAX = OFF_TAB + 2 * 4 * MATS * MP * 4;   // SwiGLU: [4 warps][MP] maxima, [3][MP] scale constants
    static constexpr int OFF_BAR = OFF_MAX + (SWIGLU ? 7 * MP * 4 : 0);
    static constexpr int NBAR = 3 * NST + 1;                     // full[NST] done[NST] empty[NST] drain
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;          // TMEM address, abort flag
    static constexpr int OFF_PRE = OFF_MISC + 8;                 // first tile, then first row of each expert
    static constexpr int smem(int G) { return OFF_PRE + 8 * (G + 1) + 768; }
    static_assert(STAGE % 1024 == 0, "swizzled tiles");
    static_assert(MATS * (MP / 4 + SB_MAX_SPLITS - 1) * 2048 <= NST * STAGE, "the exchanged sums fit in the ring");
    // CTAs that share an SM: PER_SM, or one where the experts' tables take the room of the
    // second (SwiGLU in tiles of 32 rows from 165 experts on, products in tiles of 16 from 460).
    static constexpr int per_sm(int G) { return PER_SM * (smem(G) + 1024) <= SB_SM_BYTES ? PER_SM : 1; }
    static_assert(smem(512) <= 232448, "shared memory");
    static_assert(per_sm(128) == PER_SM && NST * COLS <= TMEM && TMEM * PER_SM <= 512, "an SM's share");
};

struct SkinnyBArgs {
    ProductArgs p;
    int splits;
};

// First tile of every expert, pre[0 .. G], and behind it their first rows [0 .. G] (one
// warp).  An expert has a tile for
// each MP of its rows and each 128 weight rows; its row chunks come fastest, so
// that those that share weight rows run together.
__device__ __forceinline__ void first_tiles(const ProductArgs &a, int mp, int lane, int32_t *pre)
{
    int base = 0;
    if (lane == 0) pre[0] = 0;
    for (int g0 = 0; g0 < a.G; g0 += 32) {
        int64_t lo = 0, hi = 0;
        if (g0 + lane < a.G) expert_rows(a, g0 + lane, lo, hi);
        int sum = static_cast<int>((hi - lo + mp - 1) / mp) * a.nb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += u;
        }
        if (g0 + lane < a.G) {
            pre[g0 + lane + 1] = base + sum;
            pre[a.G + 1 + g0 + lane] = static_cast<int32_t>(lo);
            if (g0 + lane == a.G - 1) pre[2 * a.G + 1] = static_cast<int32_t>(hi);
        }
        base += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
}

// Where tile t < pre[G] lies (one whole warp, growing t).
struct SkinnyTile {
    int g0 = 0;                  // first expert of the 32 that are looked at
    int g, m0, m_end, tn;
    __device__ void seek(const ProductArgs &a, int mp, const int32_t *pre, int t, int lane)
    {
        uint32_t who;
        while ((who = __ballot_sync(0xFFFFFFFFu, g0 + lane < a.G && t < pre[g0 + lane + 1])) == 0) g0 += 32;
        g = g0 + __ffs(who) - 1;
        const int r = t - pre[g], chunks = (pre[g + 1] - pre[g]) / a.nb;
        tn = r / chunks;
        m0 = pre[a.G + 1 + g] + (r - tn * chunks) * mp;
        m_end = pre[a.G + 2 + g];
    }
};

// The bytes of four lanes' words transposed: word of lane 4 i + j, byte k <-> lane 4 i + k, byte j.
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t x, int lane)
{
    uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, x, 1);
    x = (lane & 1) ? __byte_perm(x, y, 0x3715) : __byte_perm(x, y, 0x6240);
    y = __shfl_xor_sync(0xFFFFFFFFu, x, 2);
    return (lane & 2) ? __byte_perm(x, y, 0x3276) : __byte_perm(x, y, 0x5410);
}

template <class C>
__global__ void __launch_bounds__(SB_THREADS, C::PER_SM)
product_skinny_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const SkinnyBArgs args)
{
    constexpr int MP = C::MP, NST = C::NST, MATS = C::MATS;
    constexpr bool SWIGLU = C::SWIGLU;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = sqd::smem_u32(smem);
    const ProductArgs &p = args.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = args.splits;
    const int rank = static_cast<int>(sqd::cluster_ctarank());
    if (!SWIGLU) sqd::pdl_launch_dependents();

    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto done = [&](int s) { return bar0 + 8u * (NST + s); };
    auto empty = [&](int s) { return bar0 + 8u * (2 * NST + s); };
    const uint32_t drain = bar0 + 8u * (3 * NST);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + C::OFF_MISC + 4);
    int32_t *pre = reinterpret_cast<int32_t *>(smem + C::OFF_PRE);
    auto stage = [&](int s) { return sbase + s * C::STAGE; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            sqd::mbar_init(full(s), 1);    // loads
            sqd::mbar_init(done(s), 1);    // MMAs
            sqd::mbar_init(empty(s), 4);   // epilogue warps
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
    // The first ring of weights is fetched while the previous kernel finishes, where
    // that one writes neither them nor what says which they are and has waited for
    // whoever did (ProductArgs::settled).  Experts of 4096 x 1024 x 64, one token: 34.1
    // us against 35.5 us, four: 62.9 us against 65.4 us.
    const int b_lo = p.kb * rank / S, nblk = p.kb * (rank + 1) / S - b_lo;
    const int t0 = static_cast<int>(blockIdx.x) / S;
    auto load_w = [&](int s, int b, int row) {
        sqd::mbar_arrive_expect_tx(full(s), C::STAGE);
#pragma unroll
        for (int mat = 0; mat < MATS; ++mat)
            sqd::tma_load_2d(stage(s) + mat * C::W_BYTES, &tm_w, full(s), b * BLK, row + mat * p.N);
    };
    SkinnyTile tile;
    int early = 0;
    if (warp == 0 && p.settled) {
        __syncwarp();
        first_tiles(p, MP, lane, pre);
        __syncwarp();
        if (t0 < pre[p.G]) {
            tile.seek(p, MP, pre, t0, lane);
            early = min(NST, nblk);
            if (lane == 0)
                for (int i = 0; i < early; ++i) load_w(i, b_lo + i, tile.g * MATS * p.N + tile.tn * 128);
        }
    }
    sqd::pdl_wait();  // operands, offsets and outputs may belong to the previous kernel
    if (SWIGLU) sqd::pdl_launch_dependents();   // (here: whoever starts now finds what came before this kernel complete)
    if (warp == 0 && !p.settled) first_tiles(p, MP, lane, pre);
    sqd::tc_fence_before();
    __syncthreads();
    sqd::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tiles = pre[p.G];
    // Tiles t0, t0 + step, ..: a cluster has one at most (the host's grid covers them all then).
    const int step = S > 1 ? 0x40000000 : static_cast<int>(gridDim.x);

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        // (the whole warp walks along: the next tile is looked up, which takes all lanes,
        // while the first block of this one is on its way)
        int s = 0, last = -1;
        uint32_t ph = 0, last_ph = 0;
        bool ok = true;
        if (t0 < tiles) tile.seek(p, MP, pre, t0, lane);
        for (int t = t0; ok && t < tiles; t += step) {
            const int w_row = tile.g * MATS * p.N + tile.tn * 128, x_row = tile.m0;
            for (int i = 0; i < nblk; ++i) {
                ok = __all_sync(0xFFFFFFFFu, sqd::mbar_wait_short(empty(s), ph ^ 1u, abort_flag, SITE_SB_LOAD));
                if (!ok) break;
                if (lane == 0) {
                    if (t != t0 || i >= early) load_w(s, b_lo + i, w_row);
                    sqd::tma_load_2d(stage(s) + MATS * C::W_BYTES, &tm_x, full(s), (b_lo + i) * BLK, x_row);
                }
                __syncwarp();
                last = s;
                last_ph = ph;
                if (++s == NST) { s = 0; ph ^= 1u; }
                if (i == 0 && t + step < tiles) tile.seek(p, MP, pre, t + step, lane);
            }
        }
        if (!ok && last >= 0) sqd::mbar_drain(full(last), last_ph);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        if (lane == 0) {
            constexpr uint32_t idesc = sqd::make_idesc_e4m3(128, MP);
            const uint64_t desc0 = sqd::make_sw128_desc(stage(0));   // (the ring ends below the address field's 256 KB)
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = t0; ok && t < tiles; t += step) {
                for (int i = 0; i < nblk; ++i) {
                    const uint64_t ad = desc0 + static_cast<uint64_t>(s * (C::STAGE >> 4)), bd = ad + (MATS * C::W_BYTES >> 4);
                    if (!sqd::mbar_wait_short(full(s), ph, abort_flag, SITE_SB_MMA)) { ok = false; break; }
                    sqd::tc_fence_after();
#pragma unroll
                    for (int mat = 0; mat < MATS; ++mat)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            sqd::mma_f8(tmem + s * C::COLS + mat * MP, ad + mat * (C::W_BYTES >> 4) + 2 * k, bd + 2 * k, idesc, k ? 1u : 0u);
                    sqd::mma_commit(done(s));
                    if (++s == NST) { s = 0; ph ^= 1u; }
                }
            }
            if (!ok) {
                sqd::mma_commit(drain);
                sqd::mbar_drain(drain, 0);
            }
        }
    } else {
        // ------------------------------------------------------------ sums and stores
        // (a wait that gave up does not leave the loops, so that all four warps keep
        // meeting at barrier 1; nothing is stored then)
        const int et = threadIdx.x - 64;
        const int wr = (warp & 3) * 32 + lane;   // the thread's weight row: its TMEM lane
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        float *tab = reinterpret_cast<float *>(smem + C::OFF_TAB);
        float *wmax = reinterpret_cast<float *>(smem + C::OFF_MAX);
        const int sw_up = p.nb * p.s_ld / 4;    // the up matrix's scales behind the gate's
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        int st = 0, group = 0;
        uint32_t ph = 0;
        for (int t = t0; t < tiles; t += step) {
            tile.seek(p, MP, pre, t, lane);
            const bool row_ok = et < MP && tile.m0 + et < tile.m_end;
            const float4 *sx_p = reinterpret_cast<const float4 *>(p.s_x + static_cast<int64_t>(row_ok ? tile.m0 + et : 0) * p.s_ld);
            const float4 *sw_p = reinterpret_cast<const float4 *>(p.s_w + (static_cast<int64_t>(tile.g) * MATS * p.nb + tile.tn) * p.s_ld);
            float4 sx4 = z, sw4[MATS];
            auto fetch = [&](int q) {
                sx4 = row_ok ? __ldg(sx_p + q) : z;
#pragma unroll
                for (int mat = 0; mat < MATS; ++mat) sw4[mat] = __ldg(sw_p + mat * sw_up + q);
            };
            fetch(b_lo >> 2);
            float2 acc[MATS][MP / 2];
#pragma unroll
            for (int mat = 0; mat < MATS; ++mat)
#pragma unroll
                for (int c = 0; c < MP / 2; ++c) acc[mat][c] = make_float2(0.0f, 0.0f);
            float *tq = tab;
            for (int i = 0; i < nblk; ++i) {
                const int b = b_lo + i, q = b >> 2;
                if (i == 0 || (b & 3) == 0) {
                    tq = tab + (group++ & 1) * (4 * MATS * MP);
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
                sqd::mbar_wait_short(done(st), ph, abort_flag, SITE_SB_EPI);
                sqd::tc_fence_after();
                const float4 *tb = reinterpret_cast<const float4 *>(tq + (b & 3) * MATS * MP);
#pragma unroll
                for (int ch = 0; ch < C::COLS / 16; ++ch) {
                    uint32_t v[16];
                    sqd::tmem_ld_32x32b_x16(tl + st * C::COLS + 16 * ch, v);
                    sqd::tmem_wait_ld_dep1(v);
                    if (ch + 1 == C::COLS / 16) {
                        sqd::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) sqd::mbar_arrive(empty(st));
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float4 s = tb[4 * ch + c];
                        float2 &a0 = acc[ch * 16 / MP][(ch * 16 % MP) / 2 + 2 * c], &a1 = acc[ch * 16 / MP][(ch * 16 % MP) / 2 + 2 * c + 1];
                        a0 = __ffma2_rn(make_float2(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1])), make_float2(s.x, s.y), a0);
                        a1 = __ffma2_rn(make_float2(__uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3])), make_float2(s.z, s.w), a1);
                    }
                }
                if (++st == NST) { st = 0; ph ^= 1u; }
            }
            const int n = tile.tn * 128 + wr;
            const int64_t m0 = tile.m0;
            int rows = min(MP, tile.m_end - tile.m0);        // rows of X in the tile
            if (*abort_flag) rows = 0;
            if (S == 1) {
                if constexpr (!SWIGLU) {
                    // Lanes 2 i and 2 i + 1 pair up: the even one stores row c, the odd one row c + 1, two
                    // columns each.
#pragma unroll
                    for (int c = 0; c < MP; c += 2) {
                        const float2 a = acc[0][c / 2];
                        const float o = __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? a.x : a.y, 1);
                        const __nv_bfloat162 y2 = (lane & 1) ? __floats2bfloat162_rn(o, a.y) : __floats2bfloat162_rn(a.x, o);
                        const int r = c + (lane & 1);
                        if (r < rows && n < p.N) *reinterpret_cast<__nv_bfloat162 *>(p.Y + (m0 + r) * p.ldy + (n & ~1)) = y2;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < MP / 2; ++c) {
                        const float2 gt = acc[0][c], up = acc[MATS - 1][c];
                        const float2 h = n < p.N ? silu_mul2(gt, up) : make_float2(0.0f, 0.0f);
                        acc[0][c] = h;
                        const uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(h.x)));
                        const uint32_t my = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(h.y)));
                        if (lane == 0) *reinterpret_cast<float2 *>(wmax + (warp & 3) * MP + 2 * c) = make_float2(__uint_as_float(mx), __uint_as_float(my));
                    }
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    float *consts = wmax + 4 * MP;   // of each row's scale: its inverse, its negative, the factor of tiny ones
                    if (et < MP) {
                        const CodeScale cs = code_scale(fmaxf(fmaxf(wmax[et], wmax[MP + et]), fmaxf(wmax[2 * MP + et], wmax[3 * MP + et])));
                        consts[et] = cs.inv;
                        consts[MP + et] = cs.neg;
                        consts[2 * MP + et] = cs.up;
                        if (et < rows) {
                            p.s_h[(m0 + et) * p.h_ld + tile.tn] = cs.s;
                            if (tile.tn == p.nb - 1)
                                for (int q = p.nb; q < p.h_ld; ++q) p.s_h[(m0 + et) * p.h_ld + q] = 0.0f;
                        }
                    }
                    asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
                    for (int c = 0; c < MP; c += 4) {
                        uint32_t w = 0;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 h = acc[0][c / 2 + k], inv = *reinterpret_cast<const float2 *>(consts + c + 2 * k);
                            const float2 neg = *reinterpret_cast<const float2 *>(consts + MP + c + 2 * k);
                            const float2 v = __fmul2_rn(h, *reinterpret_cast<const float2 *>(consts + 2 * MP + c + 2 * k));
                            w |= codes2(v, inv, neg) << (16 * k);
                        }
                        w = transpose_bytes(w, lane);
                        const int r = c + (lane & 3);
                        if (r < rows) *reinterpret_cast<uint32_t *>(p.H_8 + (m0 + r) * p.h_pad + tile.tn * 128 + (wr & ~3)) = w;
                    }
                }
            } else {
                // ---------------------------------------------------- exchange over the cluster
                sqd::fence_proxy_async_smem();   // the ring, filled by TMA and read by the MMAs, is written by threads below
                sqd::tc_fence_before();
                sqd::cluster_sync();             // every MMA of the cluster is complete
                // rows of X in fours, TG of them per owner: [mat][source][four][weight row]
                const int TG = (MP / 4 + S - 1) / S;
                int owner = 0, gl = 0;
#pragma unroll
                for (int c = 0; c < MP / 4; ++c) {
                    const uint32_t dst = sqd::map_to_cta(sbase + static_cast<uint32_t>(((rank * TG + gl) * 128 + wr) * 16), static_cast<uint32_t>(owner));
#pragma unroll
                    for (int mat = 0; mat < MATS; ++mat) {
                        const float2 a = acc[mat][2 * c], b2 = acc[mat][2 * c + 1];
                        sqd::st_cluster_v4(dst + static_cast<uint32_t>(mat * S * TG * 2048), __float_as_uint(a.x), __float_as_uint(a.y),
                                           __float_as_uint(b2.x), __float_as_uint(b2.y));
                    }
                    if (++gl == TG) { gl = 0; ++owner; }
                }
                sqd::cluster_sync();             // all sums delivered
                float4 *red = reinterpret_cast<float4 *>(smem);
                const int r0 = rank * TG * 4;                       // owned rows of the tile: r0 ..
                const int mine = min(4 * TG, rows - r0);
                for (int f = 0; 4 * f < mine; ++f) {
                    float4 sum[MATS];
#pragma unroll
                    for (int mat = 0; mat < MATS; ++mat) {
                        sum[mat] = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int src = 0; src < S; ++src) {
                            const float4 v = red[((mat * S + src) * TG + f) * 128 + et];
                            sum[mat].x += v.x;
                            sum[mat].y += v.y;
                            sum[mat].z += v.z;
                            sum[mat].w += v.w;
                        }
                    }
                    const int nn = tile.tn * 128 + et;
                    if constexpr (!SWIGLU) {
                        const float y[4] = {sum[0].x, sum[0].y, sum[0].z, sum[0].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (4 * f + k < mine && nn < p.N)
                                p.Y[(m0 + r0 + 4 * f + k) * p.ldy + nn] = __bfloat16_as_ushort(__float2bfloat16_rn(y[k]));
                    } else {
                        const bool in = nn < p.N;
                        const float4 gt = sum[0], up = sum[MATS - 1];
                        const float2 h01 = silu_mul2(make_float2(gt.x, gt.y), make_float2(up.x, up.y));
                        const float2 h23 = silu_mul2(make_float2(gt.z, gt.w), make_float2(up.z, up.w));
                        const float h[4] = {in ? h01.x : 0.0f, in ? h01.y : 0.0f, in ? h23.x : 0.0f, in ? h23.y : 0.0f};
                        red[f * 128 + et] = make_float4(h[0], h[1], h[2], h[3]);   // (source 0's gate sums are used up)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(h[k])));
                            if (lane == 0) wmax[(warp - 2) * MP + 4 * f + k] = __uint_as_float(m);
                        }
                    }
                }
                if constexpr (SWIGLU) {
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    const float *hs = reinterpret_cast<const float *>(smem);   // [four][column][row of the four]
                    for (int r = et >> 5; r < mine; r += 4) {       // a warp per row, four columns per lane
                        const CodeScale cs = code_scale(fmaxf(fmaxf(wmax[r], wmax[MP + r]), fmaxf(wmax[2 * MP + r], wmax[3 * MP + r])));
                        const float *h = hs + ((r >> 2) * 128 + 4 * lane) * 4 + (r & 3);
                        const float2 inv = make_float2(cs.inv, cs.inv), neg = make_float2(cs.neg, cs.neg);
                        *reinterpret_cast<uint32_t *>(p.H_8 + (m0 + r0 + r) * p.h_pad + tile.tn * 128 + 4 * lane) =
                            codes2(make_float2(h[0] * cs.up, h[4] * cs.up), inv, neg) |
                            (codes2(make_float2(h[8] * cs.up, h[12] * cs.up), inv, neg) << 16);
                        if (lane == 0) p.s_h[(m0 + r0 + r) * p.h_ld + tile.tn] = cs.s;
                        if (tile.tn == p.nb - 1 && p.nb + lane < p.h_ld) p.s_h[(m0 + r0 + r) * p.h_ld + p.nb + lane] = 0.0f;
                    }
                }
            }
        }
    }
    __syncwarp();
    if (S > 1) {
        if (warp < 2 && t0 < tiles) {   // the other warps have met there
            sqd::tc_fence_before();
            sqd::cluster_sync();
            sqd::cluster_sync();
        }
    }
    sqd::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        sqd::tc_fence_after();
        sqd::tmem_dealloc(tmem, C::TMEM);
    }
}

}  // namespace sqb
