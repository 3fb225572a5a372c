// Host side of the block-scaled FP8 calls and of the mixture-of-experts calls
// (declared in include/sq.h): argument checks and launches.  Part of
// sq_abi.cu's translation unit, whose helpers it uses.
#pragma once

namespace {

constexpr int64_t kMaxRows = 1ll << 30;

int64_t fp8b_k_pad(int64_t K) { return round_up(K, 128); }
int64_t fp8b_s_ld(int64_t K) { return round_up(K, 512) / 128; }
int64_t fp8b_row_blocks(int64_t N) { return (N + 127) / 128; }

sq_status check_K8(int64_t K, const char *name = "K")
{
    if (K < 8 || K > SQ_MAX_K || K % 8 != 0)
        return fail(SQ_ERR_INVALID_ARG, "%s=%lld must be a multiple of 8 in [8, %d]", name, (long long)K, SQ_MAX_K);
    return SQ_OK;
}

sq_status check_N8(int64_t N, const char *name = "N")
{
    if (N < 0 || N % 8 != 0 || N > kMaxRows)
        return fail(SQ_ERR_INVALID_ARG, "%s=%lld must be a non-negative multiple of 8, at most 2^30", name, (long long)N);
    return SQ_OK;
}

sq_status check_rows(int64_t M, const char *name = "M")
{
    if (M < 0 || M > kMaxRows) return fail(SQ_ERR_INVALID_ARG, "%s=%lld out of range", name, (long long)M);
    return SQ_OK;
}

sq_status check_ld(int64_t ld, int64_t n, const char *name)
{
    if (ld < n || ld % 8 != 0) return fail(SQ_ERR_INVALID_ARG, "%s must be >= %lld and a multiple of 8", name, (long long)n);
    return SQ_OK;
}

sq_status check_experts(int64_t E)
{
    if (E < 1 || E > sqm::MAX_EXPERTS)
        return fail(SQ_ERR_INVALID_ARG, "E=%lld must lie in [1, %d]", (long long)E, sqm::MAX_EXPERTS);
    return SQ_OK;
}

sq_status check_top(int64_t k)
{
    if (k < 1 || k > sqm::MAX_TOP) return fail(SQ_ERR_INVALID_ARG, "k=%lld must lie in [1, %d]", (long long)k, sqm::MAX_TOP);
    return SQ_OK;
}

// ---------------------------------------------------------------- quantizers
// (one pass at the copy rate: 8192 x 8192 33.5 us, 57344 x 8192 208 us, 3 bytes an entry
// at 6.0 and 6.8 TB/s)
sq_status prepare_fp8b_impl(const void *W, int64_t G, int64_t N, int64_t K, int64_t ldw, int64_t stride_g, void *W_8,
                            float *s_w, cudaStream_t stream)
{
    SQ_TRY(check_K8(K));
    SQ_TRY(check_N8(N));
    if (G < 0 || G > 65535) return fail(SQ_ERR_INVALID_ARG, "G=%lld must lie in [0, 65535]", (long long)G);
    SQ_TRY(check_ld(ldw, K, "ldw"));
    if (G > 1 && (stride_g < 0 || stride_g % 8 != 0)) return fail(SQ_ERR_INVALID_ARG, "stride_g must be a non-negative multiple of 8");
    if (G == 0 || N == 0) return SQ_OK;
    SQ_TRY(check_ptr(W, true, "W"));
    SQ_TRY(check_ptr(W_8, true, "W_8"));
    SQ_TRY(check_ptr(s_w, true, "s_w"));
    const int64_t nb = fp8b_row_blocks(N);
    if (nb > 65535) return fail(SQ_ERR_UNSUPPORTED, "N=%lld: more than 65535 blocks of 128 rows", (long long)N);
    DevInfo di;
    SQ_TRY(device_info(di));
    const cudaError_t e = launch_k(sqb::weight_blocks_kernel,
                                   dim3(static_cast<unsigned>(fp8b_s_ld(K)), static_cast<unsigned>(nb), static_cast<unsigned>(G)),
                                   dim3(256), 0, stream, 0u, static_cast<const uint16_t *>(W), static_cast<int>(N),
                                   static_cast<int>(K), ldw, stride_g, static_cast<int>(fp8b_k_pad(K)),
                                   static_cast<int>(fp8b_s_ld(K)), static_cast<uint8_t *>(W_8), s_w);
    return e == cudaSuccess ? SQ_OK : cuda_fail(e, "weight blocks launch");
}

bool few_warps(int64_t M, int64_t K) { return M * ((fp8b_s_ld(K) + 7) / 8) <= 64; }

// top == 0: row r of X to row r; otherwise to the rows pos[r * top ..].
sq_status quant_fp8b_impl(const void *X, int64_t M, int64_t K, int64_t ldx, const int32_t *pos, int64_t top, int64_t rows_out,
                          void *X_8, float *s_x, cudaStream_t stream)
{
    SQ_TRY(check_K8(K));
    SQ_TRY(check_rows(M));
    SQ_TRY(check_ld(ldx, K, "ldx"));
    if (M == 0 || rows_out == 0) return SQ_OK;
    SQ_TRY(check_ptr(X, true, "X"));
    SQ_TRY(check_ptr(pos, top > 0, "pos"));
    SQ_TRY(check_ptr(X_8, true, "X_8"));
    SQ_TRY(check_ptr(s_x, true, "s_x"));
    DevInfo di;
    SQ_TRY(device_info(di));
    // 1024 channels per warp; with a few warps' worth of them 256, and one copy of a row per
    // warp (8 copies of one token of 4096 channels: 5.8 us and 4.1 us).
    const bool few = few_warps(M, K);
    const int64_t tasks = M * ((fp8b_s_ld(K) * 128 + (few ? 255 : 1023)) / (few ? 256 : 1024));
    const int64_t blocks = std::min<int64_t>((tasks + sqb::QB_THREADS / 32 - 1) / (sqb::QB_THREADS / 32), 8ll * di.sms);
    const cudaError_t e = launch_k(few ? sqb::quant_kernel<1> : sqb::quant_kernel<4>,
                                   dim3(static_cast<unsigned>(blocks), few ? static_cast<unsigned>(std::max<int64_t>(1, top)) : 1u),
                                   dim3(sqb::QB_THREADS), 0, stream, 0u, static_cast<const uint16_t *>(X), M, static_cast<int>(K), ldx,
                                   static_cast<int>(fp8b_k_pad(K)), static_cast<int>(fp8b_s_ld(K)), pos, static_cast<int>(top),
                                   rows_out, static_cast<uint8_t *>(X_8), s_x);
    return e == cudaSuccess ? SQ_OK : cuda_fail(e, "block quantizer launch");
}

// ---------------------------------------------------------------- products
// 256 x 256 tiles (SwiGLU: 256 x 128 of h) on CTA pairs.
template <bool SWIGLU>
sq_status launch_pair(const DevInfo &di, const sqb::ProductArgs &a, cudaStream_t stream)
{
    constexpr int MATS = SWIGLU ? 2 : 1;
    const int64_t w_rows = static_cast<int64_t>(a.G) * MATS * a.N;
    if (w_rows > 0x7FFFFFFFll) return fail(SQ_ERR_UNSUPPORTED, "%lld weight rows", (long long)w_rows);
    CUtensorMap m_x{}, m_w{}, m_y{};
    SQ_TRY(make_map(m_x, a.X_8, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.k_pad, a.M, a.k_pad, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B));
    SQ_TRY(make_map(m_w, a.W_8, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.k_pad, w_rows, a.k_pad, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B));
    if (!SWIGLU)
        SQ_TRY(make_map(m_y, a.Y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.N, a.M, static_cast<uint64_t>(a.ldy) * 2, 64, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B));
    sqb::PairArgs pa;
    pa.p = a;
    pa.nt = SWIGLU ? a.nb : (a.nb + 1) / 2;
    const int64_t mt = (a.M + sqb::PP_BM - 1) / sqb::PP_BM;
    pa.group_m = raster_group(static_cast<int>(mt), sqb::PP_BM, 2 * a.k_pad, 0);
    const int64_t tiles = (mt + (a.offsets ? std::min<int64_t>(a.G, a.M) : 0)) * pa.nt;
    const int64_t clusters = std::min<int64_t>(tiles, di.sms / 2);
    const size_t smem = sqb::pp_smem_bytes(a.G);
    auto kern = sqb::product_pair_kernel<SWIGLU>;
    int per_sm = 0;
    SQ_TRY(kernel_setup(reinterpret_cast<const void *>(kern), sqb::PP_THREADS, smem, per_sm, "block-scaled pair set-up"));
    const cudaError_t e = launch_k(kern, dim3(static_cast<unsigned>(2 * clusters)), dim3(sqb::PP_THREADS), smem, stream, 0u, m_x,
                                   m_w, m_y, pa);
    return e == cudaSuccess ? SQ_OK : cuda_fail(e, "block-scaled pair launch");
}

// Clusters of S CTAs that the device runs at once (asked once per kernel, size and
// cluster; a GPC's SMs need not divide by S).
struct ClusterFit {
    const void *fn;
    int dev;
    size_t smem;
    unsigned S;
    int clusters;
};
std::vector<ClusterFit> g_fits;
std::mutex g_fits_mu;

sq_status cluster_fit(const void *fn, int threads, size_t smem, unsigned S, int &clusters)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lk(g_fits_mu);
    for (const ClusterFit &f : g_fits)
        if (f.fn == fn && f.dev == dev && f.smem == smem && f.S == S) {
            clusters = f.clusters;
            return SQ_OK;
        }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = S;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg)) != cudaSuccess) return cuda_fail(e, "cluster occupancy");
    g_fits.push_back({fn, dev, smem, S, clusters});
    return SQ_OK;
}

// 128 weight rows x MP rows of X, K split over clusters.
template <class C>
sq_status launch_skinny_b(const DevInfo &di, const sqb::ProductArgs &a, cudaStream_t stream)
{
    const int64_t w_rows = static_cast<int64_t>(a.G) * C::MATS * a.N;
    if (w_rows > 0x7FFFFFFFll) return fail(SQ_ERR_UNSUPPORTED, "%lld weight rows", (long long)w_rows);
    CUtensorMap m_x{}, m_w{};
    SQ_TRY(make_map(m_x, a.X_8, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.k_pad, a.M, a.k_pad, 128, C::MP, CU_TENSOR_MAP_SWIZZLE_128B));
    SQ_TRY(make_map(m_w, a.W_8, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.k_pad, w_rows, a.k_pad, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B));
    // Row chunks: at most one partial one per expert that has rows.
    const int64_t experts = a.offsets ? std::min<int64_t>(a.G, a.M) : 1;
    const int64_t tiles = (a.offsets ? a.M / C::MP + experts : (a.M + C::MP - 1) / C::MP) * a.nb;
    const size_t smem = C::smem(a.G);
    auto kern = sqb::product_skinny_kernel<C>;
    int per_sm = 0;
    SQ_TRY(kernel_setup(reinterpret_cast<const void *>(kern), sqb::SB_THREADS, smem, per_sm, "block-scaled skinny set-up"));
    // Splits: as many as let every tile run at once (experts counted with even shares of
    // the rows), and leave a CTA two blocks.
    // (CTAs that share an SM by the configuration's own arithmetic; the occupancy query
    // answers one for 110 KB of shared memory where two do run, which left half of the
    // places empty: down products of 96 tokens over 64 experts 62 us, 49 us with them)
    const int64_t cta_per_sm = C::per_sm(a.G);
    const int64_t places = cta_per_sm * di.sms;
    const int64_t at_once = a.offsets ? experts * ((a.M + experts * C::MP - 1) / (experts * C::MP)) * a.nb : tiles;
    int64_t S = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(places / at_once, sqb::SB_MAX_SPLITS), a.kb / 2));
    for (; S > 1; --S) {
        int fit = 0;
        SQ_TRY(cluster_fit(reinterpret_cast<const void *>(kern), sqb::SB_THREADS, smem, static_cast<unsigned>(S), fit));
        if (fit * cta_per_sm >= at_once) break;   // (the query counts one CTA per SM here, too)
    }
    const int64_t grid = S > 1 ? tiles * S : std::min(tiles, places);
    if (tiles > 0x3FFFFFFFll || grid > 0x7FFFFFFFll) return fail(SQ_ERR_UNSUPPORTED, "%lld tiles", (long long)tiles);
    sqb::SkinnyBArgs sa;
    sa.p = a;
    sa.splits = static_cast<int>(S);
    const cudaError_t e = launch_k(kern, dim3(static_cast<unsigned>(grid)), dim3(sqb::SB_THREADS), smem, stream,
                                   static_cast<unsigned>(S), m_x, m_w, sa);
    return e == cudaSuccess ? SQ_OK : cuda_fail(e, "block-scaled skinny launch");
}

template <bool SWIGLU>
sq_status launch_product(const sqb::ProductArgs &a, cudaStream_t stream)
{
    DevInfo di;
    SQ_TRY(device_info(di));
    // Rows per weight matrix, were they spread evenly (their counts are on the device, and
    // M counts padding too).  The figures below are of even loads; where a few experts have
    // most of the rows, either kernel is right and neither is chosen for them.
    const int64_t rows = a.offsets ? (a.M + a.G - 1) / a.G : a.M;
    // The pair kernel's 256-row tiles win where the others would read a matrix twice
    // or would hold one CTA with 128 rows on an SM, and there are tiles for the pairs:
    // above 64 rows, 80 x 8192 x 57344 is 125 us against 137 us, 128 x 8192 x 16384
    // (64 tiles) 38 us against 40 us, but 100 x 8192 x 8192 (32 tiles) 34 us against
    // 26 us; 64 experts 4096 x 1024 of 80 rows on average 87 us against 136 us.  At 64
    // rows 87 us against 78 us.  SwiGLU (64-row tiles at most): 96 rows 169 us against
    // 157 us, 128 rows 176 us against 186 us.
    if (rows > 128 || (SWIGLU ? rows > 112 : rows > 64 && a.nb * int64_t{a.G} >= 128))
        return launch_pair<SWIGLU>(di, a, stream);
    // Rows of X per tile: all of them, or fewer where even every tile split as far as
    // it goes leaves more than half of the SMs without a CTA (77 x 1000 x 1048: 9.4 us in
    // tiles of 128 rows, 5.5 us in tiles of 32; with many tiles the larger ones are
    // faster, 128 x 8192 x 8192: 29 us against 40 us in tiles of 64).
    int mp = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 || SWIGLU ? 64 : 128;
    const int64_t most = std::min<int64_t>(sqb::SB_MAX_SPLITS, std::max(1, a.kb / 2)) * a.nb * (a.offsets ? std::min<int64_t>(a.G, a.M) : 1);
    while (mp > 16 && 2 * most * ((rows + mp - 1) / mp) <= di.sms) mp /= 2;
    if (mp == 16) return launch_skinny_b<sqb::CfgSkinnyB<16, SWIGLU, SWIGLU ? 3 : 6, 2>>(di, a, stream);
    if (mp == 32) return launch_skinny_b<sqb::CfgSkinnyB<32, SWIGLU, SWIGLU ? 3 : 5, 2>>(di, a, stream);
    if constexpr (SWIGLU) return launch_skinny_b<sqb::CfgSkinnyB<64, true, 4, 1>>(di, a, stream);
    else if (mp == 64) return launch_skinny_b<sqb::CfgSkinnyB<64, false, 4, 2>>(di, a, stream);
    else return launch_skinny_b<sqb::CfgSkinnyB<128, false, 4, 1>>(di, a, stream);
}

sq_status product_args(sqb::ProductArgs &a, const void *X_8, const float *s_x, const int32_t *offsets, int64_t M, const void *W_8,
                       const float *s_w, int64_t G, int64_t N, int64_t K)
{
    SQ_TRY(check_K8(K));
    SQ_TRY(check_N8(N));
    SQ_TRY(check_rows(M));
    a = {};
    if (M == 0 || N == 0) return SQ_OK;
    SQ_TRY(check_ptr(X_8, true, "X_8"));
    SQ_TRY(check_ptr(s_x, true, "s_x"));
    SQ_TRY(check_ptr(W_8, true, "W_8"));
    SQ_TRY(check_ptr(s_w, true, "s_w"));
    a.X_8 = static_cast<const uint8_t *>(X_8);
    a.s_x = s_x;
    a.W_8 = static_cast<const uint8_t *>(W_8);
    a.s_w = s_w;
    a.offsets = offsets;
    a.M = M;
    a.G = static_cast<int>(G);
    a.N = static_cast<int>(N);
    a.k_pad = static_cast<int>(fp8b_k_pad(K));
    a.kb = a.k_pad / 128;
    a.s_ld = static_cast<int>(fp8b_s_ld(K));
    a.nb = static_cast<int>(fp8b_row_blocks(N));
    return SQ_OK;
}

sq_status gemm_fp8b_impl(const void *X_8, const float *s_x, const int32_t *offsets, int64_t M, const void *W_8, const float *s_w,
                         int64_t G, int64_t N, int64_t K, void *Y, int64_t ldy, cudaStream_t stream, bool settled = false)
{
    sqb::ProductArgs a;
    SQ_TRY(product_args(a, X_8, s_x, offsets, M, W_8, s_w, G, N, K));
    a.settled = settled;
    SQ_TRY(check_ld(ldy, N, "ldy"));
    if (M == 0 || N == 0) return SQ_OK;
    SQ_TRY(check_ptr(Y, true, "Y"));
    a.Y = static_cast<uint16_t *>(Y);
    a.ldy = ldy;
    return launch_product<false>(a, stream);
}

size_t linear_ws_bytes_fp8b(int64_t M, int64_t K)
{
    if (M <= 0) return 0;
    return static_cast<size_t>(round_up(M * fp8b_k_pad(K), 256) + round_up(M * fp8b_s_ld(K) * 4, 256));
}

sq_status linear_fp8b_impl(const void *X, int64_t M, int64_t K, int64_t ldx, const void *W_8, const float *s_w, int64_t N, void *Y,
                           int64_t ldy, void *workspace, size_t ws_bytes, cudaStream_t stream)
{
    SQ_TRY(check_K8(K));
    SQ_TRY(check_N8(N));
    SQ_TRY(check_rows(M));
    SQ_TRY(check_ld(ldx, K, "ldx"));
    SQ_TRY(check_ld(ldy, N, "ldy"));
    const size_t need = linear_ws_bytes_fp8b(M, K);
    if (ws_bytes < need) return fail(SQ_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", ws_bytes, need);
    if (M == 0 || N == 0) return SQ_OK;
    SQ_TRY(check_ptr(X, true, "X"));
    SQ_TRY(check_ptr(W_8, true, "W_8"));
    SQ_TRY(check_ptr(s_w, true, "s_w"));
    SQ_TRY(check_ptr(Y, true, "Y"));
    SQ_TRY(check_ptr(workspace, true, "workspace"));
    uint8_t *X_8 = static_cast<uint8_t *>(workspace);
    float *s_x = reinterpret_cast<float *>(X_8 + round_up(M * fp8b_k_pad(K), 256));
    SQ_TRY(quant_fp8b_impl(X, M, K, ldx, nullptr, 0, M, X_8, s_x, stream));
    return gemm_fp8b_impl(X_8, s_x, nullptr, M, W_8, s_w, 1, N, K, Y, ldy, stream, true);
}

// ---------------------------------------------------------------- experts
sq_status route_impl(const void *logits, int logits_bf16, int64_t T, int64_t E, int64_t ldl, const float *bias, int sigmoid,
                     int64_t groups, int64_t keep, int64_t group_top, int64_t k, int renorm, float scale, int32_t *ids,
                     float *weights, cudaStream_t stream)
{
    SQ_TRY(check_rows(T, "T"));
    SQ_TRY(check_experts(E));
    SQ_TRY(check_top(k));
    if (ldl < E) return fail(SQ_ERR_INVALID_ARG, "ldl must be >= E");
    if (groups < 1 || groups > sqm::MAX_GROUPS || E % groups != 0)
        return fail(SQ_ERR_INVALID_ARG, "groups=%lld must divide E and lie in [1, %d]", (long long)groups, sqm::MAX_GROUPS);
    if (keep < 1 || keep > groups) return fail(SQ_ERR_INVALID_ARG, "keep_groups must lie in [1, groups]");
    if (group_top < 1 || group_top > 2) return fail(SQ_ERR_INVALID_ARG, "group_top must be 1 or 2");
    if (k > E / groups * keep) return fail(SQ_ERR_INVALID_ARG, "k=%lld exceeds the experts of the kept groups", (long long)k);
    if (T == 0) return SQ_OK;
    SQ_TRY(check_ptr(logits, true, "logits"));
    SQ_TRY(check_ptr(bias, bias != nullptr, "bias"));
    SQ_TRY(check_ptr(ids, true, "ids"));
    SQ_TRY(check_ptr(weights, true, "weights"));
    DevInfo di;
    SQ_TRY(device_info(di));
    sqm::RouteArgs a;
    a.logits = logits;
    a.T = T;
    a.ld = ldl;
    a.bias = bias;
    a.E = static_cast<int>(E);
    a.top = static_cast<int>(k);
    a.groups = static_cast<int>(groups);
    a.keep = static_cast<int>(keep);
    a.group_top = static_cast<int>(group_top);
    a.bf16 = logits_bf16;
    // 16-byte loads: whole lanes of 4 fp32 or 8 bf16 logits, every row on a 16-byte boundary
    const int lane_logits = logits_bf16 ? 8 : 4;
    a.vec = E % (32 * lane_logits) == 0 && (E & (E - 1)) == 0 && ldl % lane_logits == 0;
    a.sigmoid = sigmoid;
    a.renorm = renorm;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    auto kern = E <= 32 ? sqm::route_kernel<1> : E <= 64 ? sqm::route_kernel<2> : E <= 128 ? sqm::route_kernel<4>
              : E <= 256 ? sqm::route_kernel<8> : sqm::route_kernel<16>;
    const cudaError_t e = launch_k(kern, dim3(static_cast<unsigned>((T + sqm::RT_WARPS - 1) / sqm::RT_WARPS)),
                                   dim3(32 * sqm::RT_WARPS), 0, stream, 0u, a);
    return e == cudaSuccess ? SQ_OK : cuda_fail(e, "route launch");
}

sq_status check_pairs(int64_t T, int64_t k)
{
    SQ_TRY(check_rows(T, "T"));
    SQ_TRY(check_top(k));
    if (T * k > kMaxRows) return fail(SQ_ERR_INVALID_ARG, "T * k=%lld out of range", (long long)(T * k));
    return SQ_OK;
}

sq_status dispatch_impl(const int32_t *ids, int64_t T, int64_t k, int64_t E, int32_t *offsets, int32_t *pos, cudaStream_t stream)
{
    SQ_TRY(check_pairs(T, k));
    SQ_TRY(check_experts(E));
    SQ_TRY(check_ptr(ids, T > 0, "ids"));
    SQ_TRY(check_ptr(offsets, true, "offsets"));
    SQ_TRY(check_ptr(pos, T > 0, "pos"));
    DevInfo di;
    SQ_TRY(device_info(di));
    const size_t smem = (static_cast<size_t>(sqm::DP_WARPS) * E + 2 * E + 1) * sizeof(int32_t);
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(sqm::DP_CTAS, T * k / sqm::DP_PAIRS));
    int per_sm = 0;
    SQ_TRY(kernel_setup(reinterpret_cast<const void *>(sqm::dispatch_kernel), 32 * sqm::DP_WARPS, smem, per_sm, "dispatch set-up"));
    const cudaError_t e = launch_k(sqm::dispatch_kernel, dim3(static_cast<unsigned>(ctas)), dim3(32 * sqm::DP_WARPS), smem, stream,
                                   static_cast<unsigned>(ctas), ids, T * k, static_cast<int>(E), offsets, pos);
    return e == cudaSuccess ? SQ_OK : cuda_fail(e, "dispatch launch");
}

sq_status swiglu_fp8b_impl(const void *X_8, const float *s_x, const int32_t *offsets, int64_t R, const void *W13_8,
                           const float *s_w13, int64_t E, int64_t I, int64_t K, void *H_8, float *s_h, cudaStream_t stream)
{
    sqb::ProductArgs a;
    SQ_TRY(check_experts(E));
    SQ_TRY(check_K8(I, "I"));
    SQ_TRY(product_args(a, X_8, s_x, offsets, R, W13_8, s_w13, E, I, K));
    if (R == 0) return SQ_OK;
    SQ_TRY(check_ptr(offsets, true, "offsets"));
    SQ_TRY(check_ptr(H_8, true, "H_8"));
    SQ_TRY(check_ptr(s_h, true, "s_h"));
    a.H_8 = static_cast<uint8_t *>(H_8);
    a.s_h = s_h;
    a.h_pad = static_cast<int>(fp8b_k_pad(I));
    a.h_ld = static_cast<int>(fp8b_s_ld(I));
    return launch_product<true>(a, stream);
}

sq_status grouped_fp8b_impl(const void *X_8, const float *s_x, const int32_t *offsets, int64_t R, const void *W_8,
                            const float *s_w, int64_t E, int64_t N, int64_t K, void *Y, int64_t ldy, cudaStream_t stream,
                            bool settled = false)
{
    SQ_TRY(check_experts(E));
    if (R > 0 && N > 0) SQ_TRY(check_ptr(offsets, true, "offsets"));
    return gemm_fp8b_impl(X_8, s_x, offsets, R, W_8, s_w, E, N, K, Y, ldy, stream, settled);
}

sq_status combine_impl(const void *Z, int64_t R, int64_t ldz, const int32_t *pos, const float *weights, int64_t T, int64_t k,
                       int64_t N, void *Y, int64_t ldy, cudaStream_t stream)
{
    SQ_TRY(check_pairs(T, k));
    SQ_TRY(check_rows(R, "R"));
    SQ_TRY(check_N8(N));
    SQ_TRY(check_ld(ldz, N, "ldz"));
    SQ_TRY(check_ld(ldy, N, "ldy"));
    if (T == 0 || N == 0) return SQ_OK;
    SQ_TRY(check_ptr(Z, R > 0, "Z"));
    SQ_TRY(check_ptr(pos, true, "pos"));
    SQ_TRY(check_ptr(weights, true, "weights"));
    SQ_TRY(check_ptr(Y, true, "Y"));
    DevInfo di;
    SQ_TRY(device_info(di));
    // small blocks where they spread over more SMs
    const int threads = T * (N / 8) <= int64_t{di.sms} * 64 ? 64 : sqm::CB_THREADS;
    const int64_t blocks = std::min<int64_t>((T * (N / 8) + threads - 1) / threads, 1ll << 30);
    auto kern = k <= 2 ? sqm::combine_kernel<2> : k <= 4 ? sqm::combine_kernel<4> : sqm::combine_kernel<8>;
    const cudaError_t e = launch_k(kern, dim3(static_cast<unsigned>(blocks)), dim3(static_cast<unsigned>(threads)), 0, stream, 0u,
                                   static_cast<const uint16_t *>(Z), R, ldz, pos, weights, T, static_cast<int>(k),
                                   static_cast<int>(N), static_cast<uint16_t *>(Y), ldy);
    return e == cudaSuccess ? SQ_OK : cuda_fail(e, "combine launch");
}

// Workspace of sq_experts_fp8b: the pairs' rows of x, of h and of the experts'
// outputs, each 256-byte aligned.
struct ExpertsLayout {
    int64_t off_pos, off_x8, off_sx, off_h8, off_sh, off_z, bytes;
    ExpertsLayout(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I)
    {
        const int64_t R = T * k;
        off_pos = round_up((E + 1) * 4, 256);
        off_x8 = off_pos + round_up(R * 4, 256);
        off_sx = off_x8 + round_up(R * fp8b_k_pad(H), 256);
        off_h8 = off_sx + round_up(R * fp8b_s_ld(H) * 4, 256);
        off_sh = off_h8 + round_up(R * fp8b_k_pad(I), 256);
        off_z = off_sh + round_up(R * fp8b_s_ld(I) * 4, 256);
        bytes = off_z + round_up(R * H * 2, 256);
    }
};

sq_status experts_fp8b_impl(const void *X, int64_t T, int64_t H, int64_t ldx, const int32_t *ids, const float *weights, int64_t k,
                            const void *W13_8, const float *s_w13, const void *W2_8, const float *s_w2, int64_t E, int64_t I,
                            void *Y, int64_t ldy, void *workspace, size_t ws_bytes, cudaStream_t stream)
{
    SQ_TRY(check_pairs(T, k));
    SQ_TRY(check_experts(E));
    SQ_TRY(check_K8(H, "H"));
    SQ_TRY(check_K8(I, "I"));
    SQ_TRY(check_ld(ldx, H, "ldx"));
    SQ_TRY(check_ld(ldy, H, "ldy"));
    if (T == 0) return SQ_OK;
    const ExpertsLayout L(T, k, E, H, I);
    if (ws_bytes < static_cast<size_t>(L.bytes))
        return fail(SQ_ERR_INVALID_ARG, "workspace of %zu bytes, %lld needed", ws_bytes, (long long)L.bytes);
    SQ_TRY(check_ptr(X, true, "X"));
    SQ_TRY(check_ptr(ids, true, "ids"));
    SQ_TRY(check_ptr(weights, true, "weights"));
    SQ_TRY(check_ptr(W13_8, true, "W13_8"));
    SQ_TRY(check_ptr(s_w13, true, "s_w13"));
    SQ_TRY(check_ptr(W2_8, true, "W2_8"));
    SQ_TRY(check_ptr(s_w2, true, "s_w2"));
    SQ_TRY(check_ptr(Y, true, "Y"));
    SQ_TRY(check_ptr(workspace, true, "workspace"));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int32_t *offsets = reinterpret_cast<int32_t *>(ws);
    int32_t *pos = reinterpret_cast<int32_t *>(ws + L.off_pos);
    uint8_t *x8 = ws + L.off_x8, *h8 = ws + L.off_h8;
    float *sx = reinterpret_cast<float *>(ws + L.off_sx), *sh = reinterpret_cast<float *>(ws + L.off_sh);
    void *Z = ws + L.off_z;
    const int64_t R = T * k;
    if (R <= sqm::DQ_PAIRS && few_warps(T, H)) {
        DevInfo di;
        SQ_TRY(device_info(di));
        const int64_t warps = T * ((fp8b_s_ld(H) * 128 + 255) / 256);
        const cudaError_t e = launch_k(sqm::dispatch_quant_kernel, dim3(static_cast<unsigned>((warps + 7) / 8), static_cast<unsigned>(k)),
                                       dim3(sqb::QB_THREADS), 0, stream, 0u, ids, static_cast<int>(T), static_cast<int>(k),
                                       static_cast<int>(E), offsets, pos, static_cast<const uint16_t *>(X), static_cast<int>(H), ldx,
                                       static_cast<int>(fp8b_k_pad(H)), static_cast<int>(fp8b_s_ld(H)), x8, sx);
        if (e != cudaSuccess) return cuda_fail(e, "dispatch and quantizer launch");
    } else {
        SQ_TRY(dispatch_impl(ids, T, k, E, offsets, pos, stream));
        SQ_TRY(quant_fp8b_impl(X, T, H, ldx, pos, k, R, x8, sx, stream));
    }
    // Z, the experts' outputs, is bf16 like every product's Y (sq_moe_gemm_fp8b and
    // sq_moe_combine take the same steps): one more rounding, half a step of each summand.
    // Against 64 bits the result is off by 0.0023 of its norm, 0.0017 of that the rounding of
    // Y itself; fp32 would write and read R * H * 2 bytes more each (4096 tokens, 8 of 64,
    // H = 4096: 0.54 GB, 82 us at the copy rate in a call of 760 us).
    SQ_TRY(swiglu_fp8b_impl(x8, sx, offsets, R, W13_8, s_w13, E, I, H, h8, sh, stream));
    // (offsets come from the dispatch, which the SwiGLU product has waited for when it lets this one start)
    SQ_TRY(grouped_fp8b_impl(h8, sh, offsets, R, W2_8, s_w2, E, H, I, Z, H, stream, true));
    return combine_impl(Z, R, H, pos, weights, T, k, H, Y, ldy, stream);
}

// Nothing may leave a C entry but its status.
template <typename F>
sq_status guarded(F &&f)
{
    try {
        g_detail.clear();
        return f();
    } catch (const std::exception &e) {
        return SQ_ERR_CUDA;
    } catch (...) {
        return SQ_ERR_CUDA;
    }
}

}  // namespace

extern "C" {

int64_t sq_k_pad_fp8b(int64_t K) { return fp8b_k_pad(K); }

int64_t sq_scale_ld_fp8b(int64_t K) { return fp8b_s_ld(K); }

sq_status sq_prepare_weights_fp8b(const void *W, int64_t G, int64_t N, int64_t K, int64_t ldw, int64_t stride_g, void *W_8,
                                  float *s_w, sq_stream_t stream)
{
    return guarded([&] { return prepare_fp8b_impl(W, G, N, K, ldw, stride_g, W_8, s_w, reinterpret_cast<cudaStream_t>(stream)); });
}

sq_status sq_quant_fp8b(const void *X, int64_t M, int64_t K, int64_t ldx, void *X_8, float *s_x, sq_stream_t stream)
{
    return guarded([&] { return quant_fp8b_impl(X, M, K, ldx, nullptr, 0, M, X_8, s_x, reinterpret_cast<cudaStream_t>(stream)); });
}

sq_status sq_gemm_fp8b(const void *X_8, const float *s_x, const void *W_8, const float *s_w, int64_t M, int64_t N, int64_t K,
                       void *Y, int64_t ldy, sq_stream_t stream)
{
    return guarded([&] {
        return gemm_fp8b_impl(X_8, s_x, nullptr, M, W_8, s_w, 1, N, K, Y, ldy, reinterpret_cast<cudaStream_t>(stream));
    });
}

size_t sq_linear_workspace_bytes_fp8b(int64_t M, int64_t K) { return linear_ws_bytes_fp8b(M, K); }

sq_status sq_linear_fp8b(const void *X, int64_t M, int64_t K, int64_t ldx, const void *W_8, const float *s_w, int64_t N, void *Y,
                         int64_t ldy, void *workspace, size_t ws_bytes, sq_stream_t stream)
{
    return guarded([&] {
        return linear_fp8b_impl(X, M, K, ldx, W_8, s_w, N, Y, ldy, workspace, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
    });
}

sq_status sq_route(const void *logits, int logits_bf16, int64_t T, int64_t E, int64_t ldl, const float *bias, int sigmoid,
                   int64_t groups, int64_t keep_groups, int64_t group_top, int64_t k, int renorm, float scale, int32_t *ids,
                   float *weights, sq_stream_t stream)
{
    return guarded([&] {
        return route_impl(logits, logits_bf16, T, E, ldl, bias, sigmoid, groups, keep_groups, group_top, k, renorm, scale, ids,
                          weights, reinterpret_cast<cudaStream_t>(stream));
    });
}

sq_status sq_moe_dispatch(const int32_t *ids, int64_t T, int64_t k, int64_t E, int32_t *offsets, int32_t *pos, sq_stream_t stream)
{
    return guarded([&] { return dispatch_impl(ids, T, k, E, offsets, pos, reinterpret_cast<cudaStream_t>(stream)); });
}

sq_status sq_moe_quant_fp8b(const void *X, int64_t T, int64_t K, int64_t ldx, const int32_t *pos, int64_t k, void *X_8, float *s_x,
                            sq_stream_t stream)
{
    return guarded([&] {
        SQ_TRY(check_pairs(T, k));
        return quant_fp8b_impl(X, T, K, ldx, pos, k, T * k, X_8, s_x, reinterpret_cast<cudaStream_t>(stream));
    });
}

sq_status sq_moe_swiglu_fp8b(const void *X_8, const float *s_x, const int32_t *offsets, int64_t R, const void *W13_8,
                             const float *s_w13, int64_t E, int64_t I, int64_t K, void *H_8, float *s_h, sq_stream_t stream)
{
    return guarded([&] {
        return swiglu_fp8b_impl(X_8, s_x, offsets, R, W13_8, s_w13, E, I, K, H_8, s_h, reinterpret_cast<cudaStream_t>(stream));
    });
}

sq_status sq_moe_gemm_fp8b(const void *X_8, const float *s_x, const int32_t *offsets, int64_t R, const void *W_8, const float *s_w,
                           int64_t E, int64_t N, int64_t K, void *Y, int64_t ldy, sq_stream_t stream)
{
    return guarded([&] {
        return grouped_fp8b_impl(X_8, s_x, offsets, R, W_8, s_w, E, N, K, Y, ldy, reinterpret_cast<cudaStream_t>(stream));
    });
}

sq_status sq_moe_combine(const void *Z, int64_t R, int64_t ldz, const int32_t *pos, const float *weights, int64_t T, int64_t k,
                         int64_t N, void *Y, int64_t ldy, sq_stream_t stream)
{
    return guarded([&] { return combine_impl(Z, R, ldz, pos, weights, T, k, N, Y, ldy, reinterpret_cast<cudaStream_t>(stream)); });
}

size_t sq_experts_workspace_bytes_fp8b(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I)
{
    if (T <= 0 || k <= 0) return 0;
    return static_cast<size_t>(ExpertsLayout(T, k, E, H, I).bytes);
}

sq_status sq_experts_fp8b(const void *X, int64_t T, int64_t H, int64_t ldx, const int32_t *ids, const float *weights, int64_t k,
                          const void *W13_8, const float *s_w13, const void *W2_8, const float *s_w2, int64_t E, int64_t I, void *Y,
                          int64_t ldy, void *workspace, size_t ws_bytes, sq_stream_t stream)
{
    return guarded([&] {
        return experts_fp8b_impl(X, T, H, ldx, ids, weights, k, W13_8, s_w13, W2_8, s_w2, E, I, Y, ldy, workspace, ws_bytes,
                                 reinterpret_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
