// Block-scaled FP8 products on CTA pairs (many rows): tcgen05 kind::f8f6f4 with
// every 128-channel block of sums scaled on its way out of tensor memory.
//
//   Y[m,n] = sum_b sx[m,b] sw[n/128,b] * D_b[m,n],   D_b = E4M3 products of block b
//
// The scales differ from block to block, so D_b cannot stay in one accumulator.
// A 256 x 256 tile's blocks alternate between two TMEM buffers of 256 columns:
// while the tensor cores fill one (4 MMAs of 32 channels), the eight epilogue
// warps of each CTA read the other and add it, times its scale, to the tile's
// sums, which live in their registers (a warp: 32 rows x 128 columns, 128 fp32
// registers a thread; a thread's row and half tile share one scale per block).
//
// Measured on a B200 at 4096 x 8192 x 8192, cycles per block of a tile: the MMAs
// alone 629 (operands in shared memory are read at 96 and written at 64 bytes per
// 128-cycle MMA and clock, so shared memory bounds them, not the 512 of the
// tensor pipe); with the sums about 825.  What the sums are made of matters:
//   - scalar fp32 and integer instructions take cycles from the tensor pipe (4 MMAs
//     went from 517 to over 800 cycles beside a loop of scalar FMAs), packed ones
//     (FFMA2) hardly do (587), so the sums are packed and free of register copies;
//   - one issuing thread's waits and commits left the pipe idle about 460 cycles
//     per block, so two warps issue alternate blocks;
//   - sixteen warps of 64 columns were slower (290 us against 252 us then, 233 us now);
//   - beside the 128 sums a thread's 232 registers do not hold all else: four words lie on
//     its stack, written once and read back in the loop (28 local stores and 5316 local
//     loads an SM in this launch, one or two loads a block, 1.4 % of what L1 takes).
//
// Warps of each CTA: 0 loads (TMA, a ring of 128-channel blocks: 128 rows of X
// and 128 rows of W per CTA), 1 and 2 issue the pair's MMAs (first CTA), 3 only
// gives its registers away, 4..11 epilogue (TMEM lane quarter w % 4, column half
// (w - 4) / 4).
// Persistent over the tiles of all experts; the rows of X and Y are the
// experts' rows one after the other, an expert's last tile is cut by rows when
// it is stored.
//
// SwiGLU form: the pair's first CTA loads gate rows and the second one up rows of
// the same 128 columns, so that a tile's halves are x G^T and x U^T of one
// 128-column block of h.  The two warps of a lane quarter exchange half of their
// sums through shared memory, each forms 64 columns of h = silu(g) u, and with
// the block's largest magnitude (both warps' maxima) writes their E4M3 codes: h
// never leaves the SM in another form.
// (64 gate and 64 up rows per CTA need no exchange of sums but two scales a block: 368
// us against 360 us for 64 experts of 512 rows, 4096 x 1024; with a sixth ring
// stage in the freed shared memory the same.)
#pragma once

#include <type_traits>

#include "sq_fp8b.cuh"
#include "sq_gemm_common.cuh"

namespace sqb {

constexpr int PP_BM = 256, PP_BN = 256;
constexpr int PP_EPI0 = 4, PP_EPI = 8;
constexpr int PP_COLS = 128;                       // tile columns per epilogue warp
constexpr int PP_REGS_IO = 40, PP_REGS_EPI = 232;  // of the 168 a thread that 12 warps are launched with: 4 * 40 + 8 * 232 = 12 * 168
constexpr int PP_THREADS = 32 * (PP_EPI0 + PP_EPI);
constexpr int PP_OPS = 5;                        // ring stages
constexpr int PP_STAGE = 256 * 128;              // bytes per CTA: 128 rows of X, 128 of W
constexpr int PP_OFF_BOX = PP_OPS * PP_STAGE;    // per epilogue warp 8 KB: two 32 x 64 bf16 boxes, or 16 x 512 B of sums
constexpr int PP_BOX = 8192;
constexpr int PP_OFF_BAR = PP_OFF_BOX + PP_EPI * PP_BOX;
constexpr int PP_NBAR = 2 * PP_OPS + 10;         // full[OPS] empty[OPS] acc_full[2] acc_empty[2] drain[2] swap[4]
constexpr int PP_OFF_MISC = PP_OFF_BAR + 8 * PP_NBAR;   // TMEM address, abort flag
constexpr int PP_OFF_OFFS = PP_OFF_MISC + 8;     // row offsets of the experts
constexpr int pp_smem_bytes(int G) { return PP_OFF_OFFS + 4 * (G + 1) + 768; }
static_assert(pp_smem_bytes(512) <= 232448, "shared memory");
static_assert(PP_OFF_BOX % 1024 == 0, "swizzled boxes");

enum : unsigned { SITE_PP_LOAD = 0x601, SITE_PP_MMA = 0x602, SITE_PP_ACC = 0x603, SITE_PP_EPI = 0x604 };

// Tiles of all experts in order: inside an expert, bands of group_m row tiles
// sweep the column tiles, so that a W tile is fetched for a whole band.
struct TileWalk {
    const int32_t *off;
    int G, nt, group_m;
    int e, base, cnt, mt;

    __device__ TileWalk(const int32_t *off_, int G_, int nt_, int group_m_)
        : off(off_), G(G_), nt(nt_), group_m(group_m_), e(-1), base(0), cnt(0), mt(0) {}

    // The expert of tile t (calls with growing t); false behind the last one.
    __device__ bool seek(int t)
    {
        while (t >= base + cnt) {
            base += cnt;
            if (++e >= G) {
                cnt = 0;
                e = G;
                return false;
            }
            mt = max(0, (off[e + 1] - off[e] + PP_BM - 1) / PP_BM);
            cnt = mt * nt;
        }
        return true;
    }
    __device__ void coords(int t, int &tmi, int &tni) const
    {
        const int idx = t - base;
        const int gsz = group_m * nt;
        const int g = idx / gsz;
        const int gm = min(mt - g * group_m, group_m);
        const int r = idx - g * gsz;
        tmi = g * group_m + r % gm;
        tni = r / gm;
    }
};

struct PairArgs {
    ProductArgs p;
    int nt, group_m;
};

// A block's sums, times the scale sv, added to the tile's; the TMEM buffer goes back
// to the MMAs (barrier `release`) once it is read.
__device__ __forceinline__ void add_block(float2 (&sums)[PP_COLS / 2], uint32_t src, float sv, int lane, uint32_t release)
{
    sqd::tc_fence_after();
    const float2 s2 = make_float2(sv, sv);
#pragma unroll
    for (int ch = 0; ch < PP_COLS / 16; ++ch) {
        uint32_t v[16];
        sqd::tmem_ld_32x32b_x16(src + 16 * ch, v);
        sqd::tmem_wait_ld_dep1(v);
        if (ch + 1 == PP_COLS / 16) {
            sqd::tc_fence_before();
            __syncwarp();
            if (lane == 0) sqd::mbar_arrive_cluster(release);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sums[8 * ch + i] = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s2, sums[8 * ch + i]);
    }
}

template <bool SWIGLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PP_THREADS, 1)
product_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_y, const PairArgs args)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];   // (the round-up covers a base that is only 256-byte aligned)
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = sqd::smem_u32(smem);
    const ProductArgs &p = args.p;
    constexpr int MATS = SWIGLU ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = sqd::cluster_ctarank();
    if (!SWIGLU) sqd::pdl_launch_dependents();

    const uint32_t bar0 = sbase + PP_OFF_BAR;
    auto full = [&](int e) { return bar0 + 8u * e; };
    auto empty = [&](int e) { return bar0 + 8u * (PP_OPS + e); };
    auto acc_full = [&](int r) { return bar0 + 8u * (2 * PP_OPS + r); };
    auto acc_empty = [&](int r) { return bar0 + 8u * (2 * PP_OPS + 2 + r); };
    auto drain = [&](uint32_t r) { return bar0 + 8u * (2 * PP_OPS + 4 + r); };
    auto swap = [&](int q) { return bar0 + 8u * (2 * PP_OPS + 6 + q); };   // SwiGLU: the two warps of lane quarter q
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + PP_OFF_MISC);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + PP_OFF_MISC + 4);
    int32_t *offs = reinterpret_cast<int32_t *>(smem + PP_OFF_OFFS);
    auto stage = [&](int e) { return sbase + e * PP_STAGE; };

    if (threadIdx.x == 0) {
        for (int e = 0; e < PP_OPS; ++e) {
            sqd::mbar_init(full(e), 2);    // each CTA's loading thread, with its bytes (first CTA's copy)
            sqd::mbar_init(empty(e), 1);   // multicast commit
        }
        for (int r = 0; r < 2; ++r) {
            sqd::mbar_init(acc_full(r), 1);              // multicast commit
            sqd::mbar_init(drain(r), 1);
            sqd::mbar_init(acc_empty(r), 2 * PP_EPI);    // both CTAs' epilogue warps (first CTA's copy)
        }
        for (int q = 0; q < 4; ++q) sqd::mbar_init(swap(q), PP_EPI / 4);
        *abort_flag = 0u;
        sqd::fence_barrier_init();
        sqd::fence_proxy_async_smem();
        sqd::prefetch_tensormap(&tm_x);
        sqd::prefetch_tensormap(&tm_w);
        if (!SWIGLU) sqd::prefetch_tensormap(&tm_y);
    }
    if (warp == 1) {
        sqd::tmem_alloc_pair(sqd::smem_u32(tmem_slot), 512);
        sqd::tmem_relinquish_pair();
    }
    sqd::pdl_wait();  // operands, offsets and outputs may belong to the previous kernel
    if (SWIGLU) sqd::pdl_launch_dependents();   // (here: whoever starts now finds what came before this kernel complete)
    for (int g = threadIdx.x; g <= p.G; g += PP_THREADS) {
        // inside the rows, whatever the offsets hold (an expert that ends before it begins has
        // no tile)
        int64_t o = p.offsets ? p.offsets[g] : (g ? p.M : 0);
        offs[g] = static_cast<int32_t>(min(max(o, int64_t(0)), p.M));
    }
    sqd::tc_fence_before();
    sqd::cluster_sync();
    sqd::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int kb = p.kb;
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    TileWalk walk(offs, p.G, args.nt, args.group_m);

    if (warp < PP_EPI0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PP_REGS_IO));
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int e = 0, last = -1;
            uint32_t ph = 0, last_ph = 0;
            bool ok = true;
            for (int t = pair; ok && walk.seek(t); t += pairs) {
                int tmi, tni;
                walk.coords(t, tmi, tni);
                const int xr = offs[walk.e] + tmi * PP_BM + static_cast<int>(rank) * 128;
                const int wr = SWIGLU ? (walk.e * 2 + static_cast<int>(rank)) * p.N + tni * 128
                                      : walk.e * p.N + tni * PP_BN + static_cast<int>(rank) * 128;
                for (int b = 0; b < kb; ++b) {
                    if (!sqd::mbar_wait_short(empty(e), ph ^ 1u, abort_flag, SITE_PP_LOAD)) { ok = false; break; }
                    const uint32_t bar = sqd::map_to_cta(full(e), 0);
                    sqd::mbar_arrive_expect_tx_cluster(bar, PP_STAGE);
                    sqd::tma_load_2d_pair(stage(e), &tm_x, bar, b * BLK, xr);
                    sqd::tma_load_2d_pair(stage(e) + 128 * 128, &tm_w, bar, b * BLK, wr);
                    last = e;
                    last_ph = ph;
                    if (++e == PP_OPS) { e = 0; ph ^= 1u; }
                }
            }
            if (!ok && last >= 0 && rank == 0) sqd::mbar_drain(full(last), last_ph);
        }
    } else if (warp < 3) {
        // ------------------------------------------------------------ MMAs (first CTA)
        // Warp 1 issues the even blocks, warp 2 the odd ones, each into its own TMEM buffer.
        if (rank == 0 && lane == 0) {
            constexpr uint32_t idesc = sqd::make_idesc_e4m3(PP_BM, PP_BN);
            const uint64_t desc0 = sqd::make_sw128_desc(stage(0));   // (the ring ends below the address field's 256 KB)
            const uint32_t r = static_cast<uint32_t>(warp - 1), d = tmem + r * PP_BN;
            int e = 0;                     // ring stage, its phase and this buffer's
            uint32_t ph = 0, free_ph = 1, g = 0;
            bool ok = true;
            for (int t = pair; ok && walk.seek(t); t += pairs) {
                for (int b = 0; b < kb; ++b, ++g) {
                    if ((g & 1u) == r) {
                        const uint64_t ad = desc0 + static_cast<uint64_t>(e * (PP_STAGE >> 4));
                        const uint64_t bd = ad + (128 * 128 >> 4);
                        if (!sqd::mbar_wait_short(full(e), ph, abort_flag, SITE_PP_MMA) ||
                            !sqd::mbar_wait_short(acc_empty(r), free_ph, abort_flag, SITE_PP_ACC)) { ok = false; break; }
                        sqd::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4; ++k) sqd::mma_f8_pair(d, ad + 2 * k, bd + 2 * k, idesc, k ? 1u : 0u);
                        sqd::mma_commit_pair_multicast(acc_full(r), 0x3);
                        sqd::mma_commit_pair_multicast(empty(e), 0x3);
                        free_ph ^= 1u;
                    }
                    if (++e == PP_OPS) { e = 0; ph ^= 1u; }
                }
            }
            if (!ok) {
                sqd::mma_commit_pair(drain(r));
                sqd::mbar_drain(drain(r), 0);
            }
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PP_REGS_EPI));
        // ------------------------------------------------------------ sums and stores
        const int quarter = warp & 3, half = (warp - PP_EPI0) >> 2;   // column half of the tile
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * PP_COLS);
        const uint32_t empty0[2] = {sqd::map_to_cta(acc_empty(0), 0), sqd::map_to_cta(acc_empty(1), 0)};
        const uint32_t box = sbase + PP_OFF_BOX + (warp - PP_EPI0) * PP_BOX;
        const int srow = static_cast<int>(rank) * 128 + quarter * 32;   // the warp's first row of the tile
        uint32_t g = 0;
        int t = pair;
        bool more = walk.seek(t), ok = true;

        // where the current tile lies, and its scales of four blocks
        int e_now = 0, tmi = 0, tni = 0, row0 = 0, row_end = 0;
        const float4 *sx_p = nullptr, *sw_p = nullptr;
        float4 sx4 = make_float4(0.f, 0.f, 0.f, 0.f), sw4 = sx4, sc = sx4;
        auto open_tile = [&]() {
            walk.coords(t, tmi, tni);
            e_now = walk.e;
            row0 = offs[e_now] + tmi * PP_BM + srow;
            row_end = offs[e_now + 1];
            const int blk = SWIGLU ? tni : tni * 2 + half;
            const bool row_ok = row0 + lane < row_end, col_ok = blk < p.nb;
            sx_p = row_ok ? reinterpret_cast<const float4 *>(p.s_x + static_cast<int64_t>(row0 + lane) * p.s_ld) : nullptr;
            sw_p = col_ok ? reinterpret_cast<const float4 *>(
                                p.s_w + (static_cast<int64_t>(e_now * MATS + (SWIGLU ? half : 0)) * p.nb + blk) * p.s_ld)
                          : nullptr;
            const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            sx4 = sx_p ? __ldg(sx_p) : z;
            sw4 = sw_p ? __ldg(sw_p) : z;
        };
        // both warps of the lane quarter have come here, and see what the other has stored
        uint32_t met = 0;
        auto meet = [&]() -> bool {
            __syncwarp();
            if (lane == 0) sqd::mbar_arrive(swap(quarter));
            const bool there = sqd::mbar_wait_short(swap(quarter), met, abort_flag, SITE_PP_EPI);
            met ^= 1u;
            return __all_sync(0xFFFFFFFFu, there);
        };
        int c_row0 = 0, c_end = 0, c_tni = 0;      // the current tile's place, once the next one is looked up
        auto next_tile = [&]() {
            c_row0 = row0;
            c_end = row_end;
            c_tni = tni;
            t += pairs;
            more = walk.seek(t);
            if (more) open_tile();
        };
        if (more) open_tile();
        while (more) {
            float2 sums[PP_COLS / 2];
#pragma unroll
            for (int i = 0; i < PP_COLS / 2; ++i) sums[i] = make_float2(0.0f, 0.0f);
            // scales of four blocks: sc, and what the next four need in flight
            const auto four_scales = [&](int b) {
                sc = make_float4(sx4.x * sw4.x, sx4.y * sw4.y, sx4.z * sw4.z, sx4.w * sw4.w);
                if (b + 4 < kb) {
                    if (sx_p) sx4 = __ldg(sx_p + (b >> 2) + 1);
                    if (sw_p) sw4 = __ldg(sw_p + (b >> 2) + 1);
                }
            };
            // (a wait that gave up does not leave the loops: a second way out would cost
            // copies of all the sums; what is added then is never stored)
            int b = 0;
            if constexpr (!SWIGLU) {       // (by four blocks: 1 to 4 % faster; the SwiGLU form has no registers for it)
#pragma unroll 1
                for (; b + 4 <= kb; b += 4) {
                    four_scales(b);
                    const float s4[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q, ++g) {
                        ok = sqd::mbar_wait_short(acc_full(g & 1u), (g >> 1) & 1u, abort_flag, SITE_PP_EPI) && ok;
                        add_block(sums, tl + (g & 1u) * PP_BN, s4[q], lane, empty0[g & 1u]);
                    }
                }
            }
#pragma unroll 1
            for (; b < kb; ++b, ++g) {
                if ((b & 3) == 0) four_scales(b);
                if (SWIGLU && b + 1 == kb) next_tile();   // (while the last block's MMAs run)
                const float sv = sc.x;
                sc = make_float4(sc.y, sc.z, sc.w, 0.0f);
                const uint32_t r = g & 1u;
                ok = sqd::mbar_wait_short(acc_full(r), (g >> 1) & 1u, abort_flag, SITE_PP_EPI) && ok;
                add_block(sums, tl + r * PP_BN, sv, lane, empty0[r]);
            }
            if (!__all_sync(0xFFFFFFFFu, ok)) break;   // (all lanes or none)
            if (!SWIGLU) next_tile();
            float acc[PP_COLS];
#pragma unroll
            for (int i = 0; i < PP_COLS / 2; ++i) {
                acc[2 * i] = sums[i].x;
                acc[2 * i + 1] = sums[i].y;
            }
            if constexpr (SWIGLU) {
                // Gate and up warp of the same rows exchange halves: the gate warp hands over its
                // columns 64.., the up warp its columns ..63; then 64 columns of both are here.
                // (one copy of the code per half: selects between the halves of acc would
                // cost four instructions per column)
                const auto finish = [&](auto up_warp) -> bool {
                    constexpr int OWN = up_warp.value ? 64 : 0, GIVE = 64 - OWN;
                    const uint32_t partner = sbase + PP_OFF_BOX + ((warp - PP_EPI0) ^ 4) * PP_BOX;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sqd::sts128(partner + i * 512 + lane * 16, __float_as_uint(acc[GIVE + 4 * i]), __float_as_uint(acc[GIVE + 4 * i + 1]),
                                    __float_as_uint(acc[GIVE + 4 * i + 2]), __float_as_uint(acc[GIVE + 4 * i + 3]));
                    if (!meet()) return false;
                    const int n0 = c_tni * 128 + OWN;
                    float mx = 0.0f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint4 o = sqd::lds128(box + i * 512 + lane * 16);
                        const float2 got[2] = {make_float2(__uint_as_float(o.x), __uint_as_float(o.y)),
                                               make_float2(__uint_as_float(o.z), __uint_as_float(o.w))};
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float2 own = make_float2(acc[OWN + 4 * i + 2 * j], acc[OWN + 4 * i + 2 * j + 1]);
                            const float2 h = up_warp.value ? silu_mul2(got[j], own) : silu_mul2(own, got[j]);
                            acc[OWN + 4 * i + 2 * j] = h.x;
                            acc[OWN + 4 * i + 2 * j + 1] = h.y;
                        }
                    }
                    if (n0 + 64 > p.N) {                 // the last tile: columns past N
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (n0 + i >= p.N) acc[OWN + i] = 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 64; ++i) mx = fmaxf(mx, fabsf(acc[OWN + i]));
                    __syncwarp();   // this warp has read its box: its rows' maxima go there
                    sqd::sts32(box + 4 * lane, __float_as_uint(mx));
                    if (!meet()) return false;
                    mx = fmaxf(mx, __uint_as_float(sqd::lds32(partner + 4 * lane)));
                    const CodeScale cs = code_scale(mx);
                    if (cs.up != 1.0f) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) acc[OWN + i] *= cs.up;
                    }
                    const int64_t m = c_row0 + lane;
                    if (m < c_end) {
                        uint8_t *out = p.H_8 + m * p.h_pad + n0;
                        const float2 inv = make_float2(cs.inv, cs.inv), neg = make_float2(cs.neg, cs.neg);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float *h = acc + OWN + 16 * i + 4 * j;
                                w[j] = codes2(make_float2(h[0], h[1]), inv, neg) | (codes2(make_float2(h[2], h[3]), inv, neg) << 16);
                            }
                            *reinterpret_cast<uint4 *>(out + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        if (!up_warp.value) {
                            p.s_h[m * p.h_ld + c_tni] = cs.s;
                            if (c_tni == p.nb - 1)
                                for (int z = p.nb; z < p.h_ld; ++z) p.s_h[m * p.h_ld + z] = 0.0f;
                        }
                    }
                    return true;
                };
                if (!(half ? finish(std::true_type()) : finish(std::false_type()))) break;
            } else {
                const int n0 = c_tni * PP_BN + half * PP_COLS;
                // the previous tile's bulk stores have read the boxes
                if (lane == 0) sqd::bulk_wait_read<0>();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 y2 = __floats2bfloat162_rn(acc[8 * i + 2 * j], acc[8 * i + 2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t *>(&y2);
                    }
                    sqd::sts128(box + (i >> 3) * 4096 + lane * 128 + (((i & 7) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
                }
                if (c_row0 + 32 <= c_end) {
                    sqd::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (n0 < p.N) sqd::tma_store_2d(&tm_y, box, n0, c_row0);
                        if (n0 + 64 < p.N) sqd::tma_store_2d(&tm_y, box + 4096, n0 + 64, c_row0);
                        sqd::bulk_commit();
                    }
                } else {
                    // the expert ends inside these 32 rows: 4 rows x 128 bytes at a time
                    __syncwarp();
                    for (int i = 0; i < 16; ++i) {
                        const int rr = (i & 7) * 4 + (lane >> 3), c = lane & 7;
                        const int n = n0 + (i >> 3) * 64 + c * 8;
                        const uint4 v = sqd::lds128(box + (i >> 3) * 4096 + rr * 128 + ((c ^ (rr & 7)) << 4));
                        if (c_row0 + rr < c_end && n < p.N)
                            *reinterpret_cast<uint4 *>(p.Y + static_cast<int64_t>(c_row0 + rr) * p.ldy + n) = v;
                    }
                    __syncwarp();
                }
            }
        }
        if (!SWIGLU && lane == 0) sqd::bulk_wait_all();
    }

    __syncwarp();
    sqd::tc_fence_before();
    sqd::cluster_sync();  // every MMA and every TMEM read of both CTAs is done
    if (warp == 1) {
        sqd::tc_fence_after();
        sqd::tmem_dealloc_pair(tmem, 512);
    }
}

}  // namespace sqb
