// libsq_fp4.cu -- the C ABI of the 4-bit microscaled formats (quantisation,
// values, product) and of the quantised key/value cache.  Like libsq.cu:
// validates arguments, sizes grids, encodes TMA tensor maps and launches; the
// contract of every entry point is in include/sq.h.
#include <cstring>
#include <type_traits>

#include "host.cuh"
#include "ptx_sm100.cuh"
#include "fp4.cuh"
#include "gemm_fp4.cuh"
#include "kvcache.cuh"

using namespace sq;

namespace sq {

cudaError_t fp4_error_words_take(unsigned int *timeout, unsigned int *bad_index)
{
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(timeout, g_error_word, sizeof(*timeout));
    if (e == cudaSuccess && *timeout != 0) e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(bad_index, kv::g_bad_index, sizeof(*bad_index));
    if (e == cudaSuccess && *bad_index != 0) e = cudaMemcpyToSymbol(kv::g_bad_index, &zero, sizeof(zero));
    return e;
}

}  // namespace sq

namespace {

inline bool valid_fmt(int f) { return f == SQ_MXFP4 || f == SQ_NVFP4; }

// The widest access (32, 16, 8 or 4 bytes, 0: single 2-byte elements) that
// every 16-element piece of rows `ld_bytes` apart allows.
inline int vec_bytes(const void *p, int64_t ld_bytes)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p) | static_cast<uint64_t>(ld_bytes);
    return (a & 31) == 0 ? 32 : (a & 15) == 0 ? 16 : (a & 7) == 0 ? 8 : (a & 3) == 0 ? 4 : 0;
}

// Blocks an SM that share a strip's rows, measured best of 2, 3, 4, 6, 8.  Two
// fit at once of either kernel for 16-bit types and four rows a thread (124 and
// 93 registers): one pass over the SMs for the quantiser, two for the dequantiser.
constexpr int QUANT_PER_SM = 2, DEQUANT_PER_SM = 4;

// Column strips of 512 x units of rows, at most `per_sm` blocks a SM.
inline dim3 strip_grid(int64_t units, int64_t cols, int per_sm)
{
    const int64_t gx = cdiv(cols, 16 * fp4::QTX);
    const int64_t target = std::max<int64_t>(1, static_cast<int64_t>(sm_count()) * per_sm / gx);
    return dim3(static_cast<unsigned>(gx), static_cast<unsigned>(std::min<int64_t>(std::min(units, target), 65535)));
}

// One row a thread instead of four where four would give two thirds of the SMs
// no block ([1021, 1000] bf16 -> NVFP4 3.9 -> 3.0 us, [200, 500] 4.2 -> 2.8; [1000,
// 2048] 3.0 and 3.2), for fp32 rows, whose four take more registers, as long as
// there are fewer than four blocks an SM ([2048, 4096] fp32 11.6 -> 8.5).  Rows
// off 16 bytes (access width 0) always go one by one.
inline bool few_units(int dt, int64_t rows, int64_t cols)
{
    const int64_t blocks = fp4::quant_units<4>(rows) * cdiv(cols, 16 * fp4::QTX);
    return dt == DT_F32 ? blocks < 4 * sm_count() : 3 * blocks < 2 * sm_count();
}

// Rows a thread, units of rows and grid of a quantiser or dequantiser whose
// rows allow accesses of `vec` bytes.
struct RowsPlan {
    int rows;
    int64_t units;
    dim3 grid;
};

inline RowsPlan plan_rows(int dt, int vec, int64_t rows, int64_t cols, int per_sm)
{
    const bool four = vec >= 16 && !few_units(dt, rows, cols);
    const int64_t units = four ? fp4::quant_units<4>(rows) : fp4::quant_units<1>(rows);
    return {four ? 4 : 1, units, strip_grid(units, cols, per_sm)};
}

// columns a quantiser covers: every byte of the scale tiles
inline int64_t quant_cols(int fmt, int64_t K) { return fp4::scale_tiles_k(fmt, K) * (fmt == SQ_MXFP4 ? 128 : 64); }

template <int DT, int VEC, int FMT>
cudaError_t launch_quant(fp4::QuantArgs a, cudaStream_t st)
{
    const RowsPlan plan = plan_rows(DT, VEC, a.rows, quant_cols(FMT, a.K), QUANT_PER_SM);
    const dim3 block(fp4::QTX, fp4::QTY);
    a.units = plan.units;
    if constexpr (VEC != 0) {
        if (plan.rows == 4) return launch_pdl(fp4::k_fp4_quant<DT, VEC, FMT, 4>, plan.grid, block, 0, st, a);
    }
    return launch_pdl(fp4::k_fp4_quant<DT, VEC, FMT, 1>, plan.grid, block, 0, st, a);
}

template <int DT, int VEC>
cudaError_t launch_quant_fmt(const fp4::QuantArgs &a, int fmt, cudaStream_t st)
{
    return fmt == SQ_MXFP4 ? launch_quant<DT, VEC, fp4::FMT_MX>(a, st) : launch_quant<DT, VEC, fp4::FMT_NV>(a, st);
}

template <int DT>
cudaError_t launch_quant_vec(const fp4::QuantArgs &a, int fmt, cudaStream_t st)
{
    const int vec = vec_bytes(a.x, a.ld * dtype_size(DT));
    if (vec == 32) return launch_quant_fmt<DT, 32>(a, fmt, st);
    if (vec == 16) return launch_quant_fmt<DT, 16>(a, fmt, st);
    return launch_quant_fmt<DT, 0>(a, fmt, st);
}

sq_status quant_fp4(const void *x, int dt, int64_t rows, int64_t K, int64_t ld, const float *s, int weight, int fmt,
                    const float *g, uint8_t *q, uint8_t *sf, sq_stream stream)
{
    if (!valid_dt(dt) || !valid_fmt(fmt) || rows < 0 || K <= 0 || ld < K) return SQ_ERR_INVALID_ARG;
    if (rows == 0) return SQ_OK;               // empty tensors have no address
    if (x == nullptr || q == nullptr || sf == nullptr) return SQ_ERR_INVALID_ARG;
    if (rows > (int64_t(1) << 40) || K > (int64_t(1) << 30) || ld > (int64_t(1) << 40)) return SQ_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(sf)) return SQ_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(x) & (dtype_size(dt) - 1)) != 0) return SQ_ERR_MISALIGNED;
    fp4::QuantArgs a{x, rows, K, ld, s, g, q, sf, 0, weight};
    const cudaStream_t st = as_stream(stream);
    const cudaError_t e = dt == SQ_F32   ? launch_quant_vec<DT_F32>(a, fmt, st)
                          : dt == SQ_F16 ? launch_quant_vec<DT_F16>(a, fmt, st)
                                         : launch_quant_vec<DT_BF16>(a, fmt, st);
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

template <int DT, int VEC>
cudaError_t launch_dequant(fp4::DequantArgs a, int fmt, cudaStream_t st)
{
    const RowsPlan plan = plan_rows(DT, VEC, a.rows, a.K, DEQUANT_PER_SM);
    const dim3 block(fp4::QTX, fp4::QTY);
    a.units = plan.units;
    auto by_format = [&](auto rows) {
        constexpr int ROWS = decltype(rows)::value;
        if (fmt == SQ_MXFP4) return launch_pdl(fp4::k_fp4_dequant<DT, VEC, fp4::FMT_MX, ROWS>, plan.grid, block, 0, st, a);
        return launch_pdl(fp4::k_fp4_dequant<DT, VEC, fp4::FMT_NV, ROWS>, plan.grid, block, 0, st, a);
    };
    if constexpr (VEC != 0) {
        if (plan.rows == 4) return by_format(std::integral_constant<int, 4>());
    }
    return by_format(std::integral_constant<int, 1>());
}

template <int DT>
cudaError_t launch_dequant_vec(const fp4::DequantArgs &a, int fmt, cudaStream_t st)
{
    const int vec = vec_bytes(a.out, a.K * dtype_size(DT));
    if (vec == 32) return launch_dequant<DT, 32>(a, fmt, st);
    if (vec == 16) return launch_dequant<DT, 16>(a, fmt, st);
    return launch_dequant<DT, 0>(a, fmt, st);
}

// ------------------------------------------------------------------ product
// Scale tiles of [rows, K] as a 3D tensor [row tiles][tiles along K][128 x
// 4 bytes]; box: kt tiles along K of nb row tiles.  Tiles outside read as 0.
bool make_scale_map(CUtensorMap *m, const void *base, int64_t ktiles, int64_t rows, uint32_t kt, uint32_t nb)
{
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(ktiles), static_cast<cuuint64_t>(cdiv(rows, 128))};
    cuuint64_t strides[2] = {fp4::SF_TILE, static_cast<cuuint64_t>(ktiles) * fp4::SF_TILE};
    cuuint32_t box[3] = {128, kt, nb};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Output map of the pair kernel's TMA stores: boxes of 32 rows x 128 bytes.
bool make_out_map128(CUtensorMap *m, void *base, int out_dt, int64_t M, int64_t N)
{
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const CUtensorMapDataType t = out_dt == SQ_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : out_dt == SQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int elt = dtype_size(out_dt);
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(N * elt)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elt), 32};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, t, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Fp4Operands {
    const void *xq, *xs, *wq, *ws;
    int64_t row_bytes, ktiles;
};

template <int BN, int CS, int FMT>
sq_status launch_fp4_swap(fp4::Fp4Params fp, const Fp4Operands &o, cudaStream_t st)
{
    using C = fp4::SwapCfg<BN, FMT>;
    constexpr uint32_t KT = fp4::SfT<FMT>::TILES;
    CUtensorMap mw, mx, mws, mxs;
    if (!make_map(&mw, o.wq, false, o.row_bytes, fp.p.N, gemm::BM)) return SQ_ERR_CUDA;
    if (!make_map(&mx, o.xq, false, o.row_bytes, fp.p.M, BN)) return SQ_ERR_CUDA;
    if (!make_scale_map(&mws, o.ws, o.ktiles, fp.p.N, KT, 1)) return SQ_ERR_CUDA;
    if (!make_scale_map(&mxs, o.xs, o.ktiles, fp.p.M, KT, 1)) return SQ_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(fp.p.tiles_r * fp.p.tiles_c * CS));
    const int per_sm = static_cast<int64_t>(grid.x) <= sm_count() ? 1 : 2;
    const int smem = C::smem_bytes(per_sm);
    fp.p.ring = C::stages(per_sm);
    auto kern = fp4::k_fp4_swap<BN, CS, FMT>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return cuda_fail(e);
    if constexpr (CS > 1)
        e = launch_pdl_cluster_smem(kern, grid, dim3(gemm::NUM_THREADS), CS, smem, st, mw, mx, mws, mxs, fp);
    else
        e = launch_pdl(kern, grid, dim3(gemm::NUM_THREADS), smem, st, mw, mx, mws, mxs, fp);
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

template <int BN, int FMT>
sq_status launch_fp4_swap_cs(const fp4::Fp4Params &fp, const Fp4Operands &o, int cs, cudaStream_t st)
{
    if (cs == 8) return launch_fp4_swap<BN, 8, FMT>(fp, o, st);
    if (cs == 4) return launch_fp4_swap<BN, 4, FMT>(fp, o, st);
    if (cs == 2) return launch_fp4_swap<BN, 2, FMT>(fp, o, st);
    return launch_fp4_swap<BN, 1, FMT>(fp, o, st);
}

// The largest cluster that leaves one CTA an SM and two K blocks a CTA: a
// second CTA an SM only adds partial sums (M = 128, N = 4096, K = 4096: 10.2 /
// 8.2 / 7.2 / 10.0 us with clusters of 1 / 2 / 4 / 8; M = 1, N = 11008: 6.4 with
// 1, 7.0 with 2; M = 1, N = 512, K = 512: 2.7 with 1, 3.3 with 2), as from about
// 90 CTAs on the weights come at HBM's rate.  Clusters of 8 only while they fill
// two thirds of the SMs: 16 of them do not fit the GPCs at once (M = 512, N =
// 512, K = 4096: 11.7 us with 16 clusters of 8).
inline int swap_cluster(int64_t tiles, int64_t num_kb)
{
    int cs = 1;
    if (!(g_inject & 2))
        while (cs < 8 && 4 * cs <= num_kb && tiles * 2 * cs <= (cs == 4 ? 2 * sm_count() / 3 : sm_count())) cs *= 2;
    return cs;
}

// How the weights-as-A kernel would run a product: tokens a tile, CTAs a
// cluster, and an estimate in us (below 0: not at all).
struct SwapPlan {
    int bn, cs;
    double us;
};

// Up to 64 tokens one tile; above, tiles of 64 or 128 tokens as long as all
// CTAs run at once (with M <= 128 the weights of one tile of 128 may take more
// waves).  The estimate, fitted to M = 64..2048, N = 64..11008, K = 256..11008 on
// B200: a start, K blocks of 256 elements, and the epilogue, which grows with
// the tile.  M = 128, N = 512, K = 512: 4.2 us with tiles of 64, 5.5 with 128;
// M = 128, N = 4096, K = 11008: 10.6 and 9.2 (clusters of 2 and 4).
inline SwapPlan plan_swap(int64_t M, int64_t N, int64_t num_kb)
{
    const int64_t tr = cdiv(N, gemm::BM);
    if (M <= 64) {
        const int bn = M <= 16 ? 16 : M <= 32 ? 32 : 64;
        return {bn, swap_cluster(tr, num_kb), 0.0};
    }
    SwapPlan best{128, 1, -1.0};
    for (const int bn : {64, 128}) {
        const int64_t tiles = tr * cdiv(M, bn);
        const int cs = swap_cluster(tiles, num_kb);
        if (tiles * cs > sm_count() && !(bn == 128 && M <= 128)) continue;
        const double us = 2.4 + (cs > 1 ? 0.9 : 0.0) + static_cast<double>(num_kb) / cs * (bn == 64 ? 0.275 : 0.31) +
                          (bn == 64 ? 1.3 : 2.6);
        if (best.us < 0 || us < best.us) best = {bn, cs, us};
    }
    return best;
}

template <int FMT>
sq_status run_fp4_swap(fp4::Fp4Params fp, const Fp4Operands &o, const SwapPlan &plan, cudaStream_t st)
{
    gemm::Params &p = fp.p;
    p.tiles_r = static_cast<int>(cdiv(p.N, gemm::BM));
    p.tiles_c = static_cast<int>(cdiv(p.M, plan.bn));
    p.num_kb = static_cast<int>(cdiv(o.row_bytes, 128));
    p.timeout_ns = g_timeout_ns;
    p.inject = g_inject & 1;
    if (plan.bn == 16) return launch_fp4_swap_cs<16, FMT>(fp, o, plan.cs, st);
    if (plan.bn == 32) return launch_fp4_swap_cs<32, FMT>(fp, o, plan.cs, st);
    if (plan.bn == 64) return launch_fp4_swap_cs<64, FMT>(fp, o, plan.cs, st);
    return launch_fp4_swap_cs<128, FMT>(fp, o, plan.cs, st);
}

// How CTA pairs would run it: tile columns and an estimate in us, the start
// included.  Measured on B200 over M = 129..4096, N = 1024..28672, K =
// 1024..11008: waves x (K blocks x time a block + time a tile).  A K block costs
// a narrow tile almost what it costs a wide one, so narrow tiles pay where they
// save a wave: M = 512, N = 12288, K = 4096 takes 16.7 / 14.9 / 19.0 us with 256
// / 192 / 128 columns, M = 1024, N = 4096, K = 4096 11.4 / 14.8 / 14.7, M = 256,
// N = 4096, K = 1024 7.1 / 6.5 / 6.1.
struct PairPlan {
    int bn;
    double us;
};

inline PairPlan plan_pair(int64_t M, int64_t N, int64_t num_kb)
{
    const int64_t clusters = std::max(1, sm_count() / 2);
    const int widths[3] = {256, 192, 128};
    const double per_kb[3] = {0.35, 0.285, 0.275}, per_tile[3] = {1.1, 0.75, 0.35};
    PairPlan best{256, -1.0};
    for (int i = 0; i < 3; ++i) {
        const int64_t tiles = cdiv(M, 2 * gemm::BM) * cdiv(N, widths[i]);
        const double us = 4.55 + static_cast<double>(cdiv(tiles, clusters)) * (static_cast<double>(num_kb) * per_kb[i] + per_tile[i]);
        if (best.us < 0 || us < best.us) best = {widths[i], us};
    }
    return best;
}

template <int BN, int FMT>
sq_status launch_fp4_pair(fp4::Fp4Params fp, const Fp4Operands &o, cudaStream_t st)
{
    using C = fp4::Pair4Cfg<BN, FMT>;
    gemm::Params &p = fp.p;
    CUtensorMap ma, mb, mas, mbs, mo;
    if (!make_map(&ma, o.xq, false, o.row_bytes, p.M, gemm::BM)) return SQ_ERR_CUDA;
    if (!make_map(&mb, o.wq, false, o.row_bytes, p.N, BN / 2)) return SQ_ERR_CUDA;
    const uint32_t kt = fp4::SfT<FMT>::TILES;
    if (!make_scale_map(&mas, o.xs, o.ktiles, p.M, kt, 1)) return SQ_ERR_CUDA;
    if (!make_scale_map(&mbs, o.ws, o.ktiles, p.N, kt, C::NB)) return SQ_ERR_CUDA;
    std::memset(&mo, 0, sizeof(mo));
    // TMA stores need 16-byte row strides and base
    fp.direct = !aligned16(p.out) || (static_cast<int64_t>(p.N) * dtype_size(p.out_dt)) % 16 != 0;
    if (!fp.direct && !make_out_map128(&mo, p.out, p.out_dt, p.M, p.N)) return SQ_ERR_CUDA;
    p.num_kb = static_cast<int>(cdiv(o.row_bytes, 128));
    const int64_t tr = cdiv(p.M, 2 * gemm::BM), tc = cdiv(p.N, BN);
    if (tr * tc >= (int64_t(1) << 31)) return SQ_ERR_UNSUPPORTED;
    p.tiles_r = static_cast<int>(tr);
    p.tiles_c = static_cast<int>(tc);
    p.num_units = static_cast<int>(tr * tc);
    p.timeout_ns = g_timeout_ns;
    p.inject = g_inject & 1;
    auto kern = fp4::k_fp4_pair<BN, FMT>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), C::SMEM_BYTES);
    if (e != cudaSuccess) return cuda_fail(e);
    int max_clusters = 0;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        max_clusters = kinfo(reinterpret_cast<const void *>(kern)).clusters;
    }
    if (max_clusters == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (sm_count() / 2), 1, 1);
        cfg.blockDim = dim3(fp4::PAIR_THREADS, 1, 1);
        cfg.dynamicSmemBytes = C::SMEM_BYTES;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void *>(kern), &cfg) != cudaSuccess || n <= 0)
            n = sm_count() / 2;
        cudaGetLastError();
        max_clusters = n;
        std::lock_guard<std::mutex> lk(g_mu);
        kinfo(reinterpret_cast<const void *>(kern)).clusters = n;
    }
    const int clusters = static_cast<int>(std::min<int64_t>(p.num_units, max_clusters));
    e = launch_pdl(kern, dim3(2 * clusters), dim3(fp4::PAIR_THREADS), C::SMEM_BYTES, st, ma, mb, mas, mbs, mo, fp);
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

// CTA pairs with tiles of bn columns, or the weights-as-A kernel (cs CTAs a cluster).
struct LinearPlan {
    bool pairs;
    int bn;
    SwapPlan swap;
};

inline LinearPlan plan_linear(int64_t M, int64_t N, int64_t num_kb)
{
    const SwapPlan swap = plan_swap(M, N, num_kb);
    if (M <= 128) return {false, swap.bn, swap};
    const PairPlan pair = plan_pair(M, N, num_kb);
    if (swap.us >= 0 && swap.us < pair.us) return {false, swap.bn, swap};
    return {true, pair.bn, swap};
}

template <int FMT>
sq_status dispatch_fp4(const fp4::Fp4Params &fp, const Fp4Operands &o, cudaStream_t st)
{
    const LinearPlan plan = plan_linear(fp.p.M, fp.p.N, cdiv(o.row_bytes, 128));
    if (!plan.pairs) return run_fp4_swap<FMT>(fp, o, plan.swap, st);
    switch (plan.bn) {
    case 256: return launch_fp4_pair<256, FMT>(fp, o, st);
    case 192: return launch_fp4_pair<192, FMT>(fp, o, st);
    default: return launch_fp4_pair<128, FMT>(fp, o, st);
    }
}

// ------------------------------------------------------------------ key/value cache
inline bool valid_kv(int f) { return f == SQ_KV_INT8 || f == SQ_KV_FP8 || f == SQ_KV_MXFP4; }

// log2 of the lanes of a warp that share a row of D elements, 16 a lane
inline int lanes_log2(int D)
{
    int l = 1;                                  // two lanes hold an MXFP4 block
    while (l < 5 && (16 << l) < D) ++l;
    return l;
}

constexpr int KV_READ_WARPS = 16;               // warps an SM below which a token's heads are split over warps

// Steps a warp and chunks of 16 elements a lane of a write: several steps once
// that leaves every SM its 64 warps.
struct WritePlan {
    int steps, chunks;
};

inline WritePlan plan_write(int64_t T, int64_t H, int64_t D)
{
    if (D > 512) return {1, 2};
    const int64_t steps = cdiv(T * H, 32 >> lanes_log2(static_cast<int>(D)));      // of a warp, for keys and again for values
    return {2 * steps >= static_cast<int64_t>(kv::TOKENS) * 64 * sm_count() ? kv::TOKENS : 1, 1};
}

// Rows end to end where a warp a token would leave lanes idle or have one
// group of heads in flight: 1 head of 64 414 -> 60 us (45 at the copy rate), 2
// of 128 107 -> 58, 5 of 128 59 -> 48; 8 of 128 stay a warp a token (69 us
// against 73 for 75 k tokens, 2.7 against 3.4 for 64).  Else 2^part_log2 warps
// a token: more than one while the heads allow and the SMs are not full.
struct ReadPlan {
    bool by_rows;
    int part_log2;
};

inline ReadPlan plan_read(int64_t total, int64_t H, int64_t D)
{
    const int ll = lanes_log2(static_cast<int>(D));
    const int64_t groups = cdiv(H, 32 >> ll);
    if (D <= 512 && ((16 << ll) != D || H % (32 >> ll) != 0 || groups < 2)) return {true, 0};
    int part = 0;
    while ((int64_t(2) << part) <= groups && (total << part) < static_cast<int64_t>(KV_READ_WARPS) * sm_count()) ++part;
    return {false, part};
}

// Calls launch(type, format, access width) with all three as compile-time
// constants (width 0: narrower than 16 bytes).
template <typename F> cudaError_t kv_dispatch(int dt, int fmt, int vec, F &&launch)
{
    auto width = [&](auto d, auto f) -> cudaError_t {
        if (vec == 32) return launch(d, f, std::integral_constant<int, 32>());
        if (vec == 16) return launch(d, f, std::integral_constant<int, 16>());
        return launch(d, f, std::integral_constant<int, 0>());
    };
    auto format = [&](auto d) -> cudaError_t {
        if (fmt == SQ_KV_INT8) return width(d, std::integral_constant<int, kv::KV_INT8>());
        if (fmt == SQ_KV_FP8) return width(d, std::integral_constant<int, kv::KV_FP8>());
        return width(d, std::integral_constant<int, kv::KV_MXFP4>());
    };
    if (dt == SQ_F32) return format(std::integral_constant<int, DT_F32>());
    if (dt == SQ_F16) return format(std::integral_constant<int, DT_F16>());
    return format(std::integral_constant<int, DT_BF16>());
}

// ceil(2^63 / d): the high word of (2 n) * inverse63(d) is n / d as long as n * d < 2^63
inline uint64_t inverse63(int64_t d) { return ((uint64_t(1) << 63) + static_cast<uint64_t>(d) - 1) / static_cast<uint64_t>(d); }

sq_status check_kv(int fmt, int dt, int64_t H, int64_t D)
{
    if (!valid_kv(fmt) || !valid_dt(dt) || H <= 0 || D <= 0) return SQ_ERR_INVALID_ARG;
    if (D > kv::MAX_D || H > 65536) return SQ_ERR_UNSUPPORTED;
    return SQ_OK;
}

}  // namespace

extern "C" {

size_t sq_fp4_code_bytes(int64_t K) { return K > 0 ? static_cast<size_t>(fp4::code_row_bytes(K)) : 0; }

size_t sq_fp4_scale_bytes(sq_fp4_format fmt, int64_t rows, int64_t K)
{
    if (!valid_fmt(fmt) || rows <= 0 || K <= 0) return 0;
    return static_cast<size_t>(cdiv(rows, 128)) * static_cast<size_t>(fp4::scale_tiles_k(fmt, K)) * fp4::SF_TILE;
}

sq_status sq_smooth_scales_nvfp4(const float *act_max, const float *w_max, int64_t K, float alpha, float *s,
                                 float *g_act, float *g_w, sq_stream stream)
{
    const sq_status r = sq_smooth_scales(act_max, w_max, K, alpha, s, nullptr, stream);
    if (r != SQ_OK || (g_act == nullptr && g_w == nullptr)) return r;
    const cudaError_t e = launch_pdl(fp4::k_nvfp4_scales, dim3(1), dim3(1024), 0, as_stream(stream), act_max, w_max, K,
                                     static_cast<const float *>(s), g_act, g_w);
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

sq_status sq_quant_weight_fp4(const void *w, sq_dtype dt, int64_t N, int64_t K, const float *s, sq_fp4_format fmt,
                              const float *g, uint8_t *wq4, uint8_t *w_sf, sq_stream stream)
{
    return quant_fp4(w, dt, N, K, K, s, 1, fmt, g, wq4, w_sf, stream);
}

sq_status sq_smooth_quant_act_fp4(const void *x, sq_dtype dt, int64_t M, int64_t K, int64_t ld, const float *s,
                                  sq_fp4_format fmt, const float *g, uint8_t *xq4, uint8_t *x_sf, sq_stream stream)
{
    return quant_fp4(x, dt, M, K, ld, s, 0, fmt, g, xq4, x_sf, stream);
}

sq_status sq_dequant_fp4(const uint8_t *q4, const uint8_t *sf, sq_fp4_format fmt, int64_t rows, int64_t K,
                         const float *g, sq_dtype out_dt, void *out, sq_stream stream)
{
    if (!valid_fmt(fmt) || !valid_dt(out_dt) || rows < 0 || K <= 0) return SQ_ERR_INVALID_ARG;
    if (rows == 0) return SQ_OK;
    if (q4 == nullptr || sf == nullptr || out == nullptr) return SQ_ERR_INVALID_ARG;
    if (rows > (int64_t(1) << 40) || K > (int64_t(1) << 30)) return SQ_ERR_UNSUPPORTED;
    if (!aligned16(q4) || !aligned16(sf)) return SQ_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(out) & (dtype_size(out_dt) - 1)) != 0) return SQ_ERR_MISALIGNED;
    fp4::DequantArgs a{q4, sf, rows, K, g, out, 0};
    const cudaStream_t st = as_stream(stream);
    const cudaError_t e = out_dt == SQ_F32   ? launch_dequant_vec<DT_F32>(a, fmt, st)
                          : out_dt == SQ_F16 ? launch_dequant_vec<DT_F16>(a, fmt, st)
                                             : launch_dequant_vec<DT_BF16>(a, fmt, st);
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

sq_status sq_linear_fp4(const uint8_t *xq4, const uint8_t *x_sf, const uint8_t *wq4, const uint8_t *w_sf,
                        sq_fp4_format fmt, int64_t M, int64_t N, int64_t K, const float *g_act, const float *g_w,
                        const void *bias, sq_dtype out_dt, void *y, sq_stream stream)
{
    if (!valid_fmt(fmt) || !valid_dt(out_dt) || M < 0 || N <= 0 || K <= 0) return SQ_ERR_INVALID_ARG;
    if (M == 0) return SQ_OK;
    if (xq4 == nullptr || x_sf == nullptr || wq4 == nullptr || w_sf == nullptr || y == nullptr) return SQ_ERR_INVALID_ARG;
    if (M > (int64_t(1) << 30) || N > (int64_t(1) << 30) || K > (int64_t(1) << 30)) return SQ_ERR_UNSUPPORTED;
    if (!aligned16(xq4) || !aligned16(x_sf) || !aligned16(wq4) || !aligned16(w_sf)) return SQ_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(y) & (dtype_size(out_dt) - 1)) != 0 ||
        (reinterpret_cast<uintptr_t>(bias) & (dtype_size(out_dt) - 1)) != 0)
        return SQ_ERR_MISALIGNED;
    fp4::Fp4Params fp{};
    gemm::Params &p = fp.p;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.bias = bias;
    p.out = y;
    p.out_dt = out_dt;
    fp.g_act = fmt == SQ_NVFP4 ? g_act : nullptr;
    fp.g_w = fmt == SQ_NVFP4 ? g_w : nullptr;
    g_fp4_launched.store(true);
    const Fp4Operands o{xq4, x_sf, wq4, w_sf, fp4::code_row_bytes(K), fp4::scale_tiles_k(fmt, K)};
    const cudaStream_t st = as_stream(stream);
    return fmt == SQ_MXFP4 ? dispatch_fp4<fp4::FMT_MX>(fp, o, st) : dispatch_fp4<fp4::FMT_NV>(fp, o, st);
}

sq_status sq_debug_linear_fp4_plan(int64_t M, int64_t N, int64_t K, int *plan)
{
    if (M <= 0 || N <= 0 || K <= 0 || plan == nullptr) return SQ_ERR_INVALID_ARG;
    const LinearPlan p = plan_linear(M, N, cdiv(fp4::code_row_bytes(K), 128));
    plan[0] = p.pairs ? 1 : 0;
    plan[1] = p.bn;
    plan[2] = p.pairs ? 2 : p.swap.cs;
    return SQ_OK;
}

sq_status sq_debug_rows_fp4_plan(int values, int fmt, sq_dtype dt, int vec, int64_t rows, int64_t K, int *plan)
{
    if (!valid_fmt(fmt) || !valid_dt(dt) || rows <= 0 || K <= 0 || plan == nullptr) return SQ_ERR_INVALID_ARG;
    const RowsPlan p = plan_rows(dt, vec, rows, values ? K : quant_cols(fmt, K), values ? DEQUANT_PER_SM : QUANT_PER_SM);
    plan[0] = p.rows;
    plan[1] = static_cast<int>(std::min<int64_t>(cdiv(p.units, p.grid.y), 1 << 30));
    return SQ_OK;
}

sq_status sq_debug_kv_plan(int64_t rows, int64_t H, int64_t D, int *plan)
{
    const sq_status r = check_kv(SQ_KV_INT8, SQ_F32, H, D);
    if (r != SQ_OK) return r;
    if (rows <= 0 || rows > (int64_t(1) << 31) || plan == nullptr) return SQ_ERR_INVALID_ARG;
    const WritePlan w = plan_write(rows, H, D);
    const ReadPlan d = plan_read(rows, H, D);
    plan[0] = w.steps;
    plan[1] = w.chunks;
    plan[2] = d.by_rows ? 1 : 0;
    plan[3] = d.by_rows ? 0 : 1 << d.part_log2;
    return SQ_OK;
}

size_t sq_kv_row_bytes(sq_kv_format fmt, int64_t D)
{
    return valid_kv(fmt) && D > 0 && D <= kv::MAX_D ? static_cast<size_t>(kv::row_bytes(fmt, static_cast<int>(D))) : 0;
}

size_t sq_kv_scale_bytes(sq_kv_format fmt, int64_t D)
{
    return valid_kv(fmt) && D > 0 && D <= kv::MAX_D ? static_cast<size_t>(kv::scale_bytes(fmt, static_cast<int>(D))) : 0;
}

sq_status sq_kv_cache_write(const void *k, const void *v, sq_dtype dt, int64_t T, int64_t H, int64_t D, int64_t k_ld,
                            int64_t v_ld, const int64_t *slots, sq_kv_format fmt, int64_t num_slots, void *k_cache,
                            void *k_scale, void *v_cache, void *v_scale, sq_stream stream)
{
    const sq_status r = check_kv(fmt, dt, H, D);
    if (r != SQ_OK) return r;
    if (T < 0 || k_ld < H * D || v_ld < H * D || num_slots < 0) return SQ_ERR_INVALID_ARG;
    if (T == 0) return SQ_OK;
    if (k == nullptr || v == nullptr || slots == nullptr) return SQ_ERR_INVALID_ARG;
    // a cache without slots has no address, and none of it is accessed
    if (num_slots > 0 && (k_cache == nullptr || k_scale == nullptr || v_cache == nullptr || v_scale == nullptr))
        return SQ_ERR_INVALID_ARG;
    if (T > (int64_t(1) << 31) || num_slots > (int64_t(1) << 40) || k_ld > (int64_t(1) << 32) || v_ld > (int64_t(1) << 32))
        return SQ_ERR_UNSUPPORTED;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) || !aligned16(v_scale))
        return SQ_ERR_MISALIGNED;
    if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & (dtype_size(dt) - 1)) != 0 ||
        (reinterpret_cast<uintptr_t>(slots) & 7) != 0)
        return SQ_ERR_MISALIGNED;
    const int ll = lanes_log2(static_cast<int>(D));
    g_fp4_launched.store(true);
    kv::WriteArgs a{k, v, T, k_ld, v_ld, num_slots, slots, static_cast<uint8_t *>(k_cache),
                    static_cast<uint8_t *>(v_cache), k_scale, v_scale, static_cast<int>(H), static_cast<int>(D), ll, 0,
                    inverse63(H)};
    const WritePlan plan = plan_write(T, H, D);
    const int64_t warps = 2 * cdiv(cdiv(T * H, 32 >> ll), plan.steps), blocks = cdiv(warps, kv::WARPS);
    if (blocks >= (int64_t(1) << 31)) return SQ_ERR_UNSUPPORTED;
    const int es = dtype_size(dt);
    a.vec = std::min(vec_bytes(k, (k_ld * es) | (D * es)), vec_bytes(v, (v_ld * es) | (D * es)));
    const cudaStream_t st = as_stream(stream);
    const cudaError_t e = kv_dispatch(dt, fmt, a.vec, [&](auto d, auto f, auto w) {
        constexpr int DT = decltype(d)::value, FMT = decltype(f)::value, VEC = decltype(w)::value;
        const dim3 grid(static_cast<unsigned>(blocks)), block(kv::WARPS * 32);
        if (plan.chunks == 2) return launch_pdl(kv::k_kv_write<DT, FMT, VEC, 2, 1>, grid, block, 0, st, a);
        if (plan.steps > 1) return launch_pdl(kv::k_kv_write<DT, FMT, VEC, 1, kv::TOKENS>, grid, block, 0, st, a);
        return launch_pdl(kv::k_kv_write<DT, FMT, VEC, 1, 1>, grid, block, 0, st, a);
    });
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

sq_status sq_kv_cache_read(sq_kv_format fmt, const void *k_cache, const void *k_scale, const void *v_cache,
                           const void *v_scale, int64_t num_pages, int64_t page_size, int64_t H, int64_t D,
                           const int32_t *table, int64_t B, int64_t max_pages, const int32_t *cu_rows,
                           const int32_t *starts, int64_t total, sq_dtype out_dt, void *k_out, void *v_out,
                           sq_stream stream)
{
    const sq_status r = check_kv(fmt, out_dt, H, D);
    if (r != SQ_OK) return r;
    if (num_pages < 0 || page_size <= 0 || B < 0 || max_pages < 0 || total < 0) return SQ_ERR_INVALID_ARG;
    if (total == 0 || B == 0) return SQ_OK;
    if (cu_rows == nullptr || k_out == nullptr || v_out == nullptr) return SQ_ERR_INVALID_ARG;
    // a cache without pages, a table without columns: no address, no access
    if (num_pages > 0 && (k_cache == nullptr || k_scale == nullptr || v_cache == nullptr || v_scale == nullptr))
        return SQ_ERR_INVALID_ARG;
    if (max_pages > 0 && table == nullptr) return SQ_ERR_INVALID_ARG;
    if (num_pages >= (int64_t(1) << 31) || page_size >= (int64_t(1) << 31) || B >= (int64_t(1) << 30) ||
        max_pages >= (int64_t(1) << 31) || total >= (int64_t(1) << 31))
        return SQ_ERR_UNSUPPORTED;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) || !aligned16(v_scale))
        return SQ_ERR_MISALIGNED;
    if (((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & (dtype_size(out_dt) - 1)) != 0 ||
        ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(cu_rows) |
          reinterpret_cast<uintptr_t>(starts)) & 3) != 0)
        return SQ_ERR_MISALIGNED;
    const int ll = lanes_log2(static_cast<int>(D));
    g_fp4_launched.store(true);
    kv::ReadArgs a{static_cast<const uint8_t *>(k_cache), static_cast<const uint8_t *>(v_cache), k_scale, v_scale,
                   num_pages, max_pages, table, cu_rows, starts, total, k_out, v_out, static_cast<int>(B),
                   static_cast<int>(H), static_cast<int>(D), static_cast<int>(cdiv(H, 32 >> ll)),
                   static_cast<int>(page_size), ll, 0, 0, 0, 0, static_cast<int>(cdiv(D, 16))};
    const int es = dtype_size(out_dt);
    a.vec = std::min(vec_bytes(k_out, D * es), vec_bytes(v_out, D * es));
    const cudaStream_t st = as_stream(stream);
    a.page_inv = inverse63(page_size);
    a.head_inv = inverse63(H);
    const ReadPlan plan = plan_read(total, H, D);
    a.part_log2 = plan.part_log2;
    const int64_t warps = plan.by_rows ? cdiv(total * H, 2 * (32 / a.lanes)) : total << a.part_log2;
    const int64_t blocks = cdiv(warps, kv::WARPS);
    if (blocks >= (int64_t(1) << 31)) return SQ_ERR_UNSUPPORTED;
    const cudaError_t e = kv_dispatch(out_dt, fmt, a.vec, [&](auto d, auto f, auto w) {
        constexpr int DT = decltype(d)::value, FMT = decltype(f)::value, VEC = decltype(w)::value;
        const dim3 grid(static_cast<unsigned>(blocks)), block(kv::WARPS * 32);
        if (plan.by_rows) return launch_pdl(kv::k_kv_read_rows<DT, FMT, VEC>, grid, block, 0, st, a);
        return launch_pdl(kv::k_kv_read<DT, FMT, VEC>, grid, block, 0, st, a);
    });
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

}  // extern "C"
