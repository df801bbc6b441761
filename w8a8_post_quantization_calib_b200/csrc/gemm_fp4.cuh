// gemm_fp4.cuh -- the product of 4-bit microscaled operands on the block-scaled
// tensor cores of sm_100a:
//
//   acc[m, n] = sum_b sx[m, b] * sw[n, b] * sum_{k in b} x[m, k] * w[n, k]     (b: blocks along K)
//   y[m, n]   = RN_out(fmaf(acc, fl(g_act * g_w), bias[n]))
//
// tcgen05.mma kind::mxf4 (E8M0 scales, blocks of 32) or kind::mxf4nvf4 (E4M3
// scales, blocks of 16): 64 elements of K an instruction, packed two a byte,
// so an operand tile is the same 128-byte-swizzled K-major tile as for the
// 8-bit kernels with twice the elements.  The scales are read from tensor
// memory: a scale tile (128 rows x 4 blocks, 512 bytes, laid out as in
// fp4.cuh) comes into shared memory by TMA and takes 4 TMEM columns (row r at
// lane r % 32, column r / 32, replicated to the four lane quarters).
//
//   k_fp4_swap (M <= 128, or few tiles): the weights fill the 128-row MMA; a
//     cluster of CS CTAs shares a tile's K range.
//     Scales go to TMEM by tcgen05.cp: issued by the MMA's thread, executed in
//     order with the MMAs, no barrier.  Roles and barriers are gemm.cuh's.
//   k_fp4_pair: CTA pairs (cta_group::2), 256 x BN tiles.  Each CTA
//     loads its 128 rows of A and BN/2 rows of B, its rows' A scales and all
//     BN rows' B scales (each SM scales its own 128 x BN accumulator).  Four
//     more warps bring the scales from their own shared-memory ring to TMEM
//     (tcgen05.st): 12 scale tiles a K block of NVFP4 (6 of MXFP4) take 0.57
//     us by tcgen05.cp, in the tensor pipe and in turn with the block's 0.29 us
//     of MMAs.  M = 8192, N = 28672, K = 8192: 1165 -> 724 us (NVFP4), 850 ->
//     708 us (MXFP4), then bound by power (5.3 PFLOP/s at ~1.5 GHz; 6.3 on
//     all-zero codes, at 1965 MHz).
#pragma once

#include <type_traits>

#include "fp4.cuh"
#include "gemm.cuh"

namespace sq {
namespace ptx {

// True in one lane of a converged warp, the same one at every call.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// Arrive on a barrier of any CTA of the cluster without publishing writes to
// memory: for work in tensor memory (reads or writes that tcgen05.wait has
// seen complete, ordered by the tcgen05 fences around the barrier) and for
// buffers that asynchronous operations have finished with.  mbar_arrive_cluster
// publishes this thread's writes at cluster scope, which takes ~0.8 us.
__device__ __forceinline__ void mbar_arrive_plain(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// 16-byte store to shared memory of a CTA of this cluster, counted as 16
// transaction bytes on that CTA's barrier (both addresses from mapa).
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t bar, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(addr),
                 "r"(bar), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// All threads of the cluster meet; no memory is published.
__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

}  // namespace ptx

namespace fp4 {

using gemm::BKB;
using gemm::BM;
using gemm::ERR_DRAIN;
using gemm::ERR_EPI;
using gemm::ERR_MMA;
using gemm::ERR_PRODUCER;
using gemm::NUM_THREADS;
using gemm::Params;
using gemm::STG_BYTES;

// Scale tiles of a 128-byte K block (256 elements), and MMAs that share one.
template <int FMT> struct SfT {
    static constexpr int TILES = 256 / FmtT<FMT>::TILE_K;          // MXFP4 2, NVFP4 4
    static constexpr int MMAS = 4 / TILES;
};

// The two factors besides the block scales, fl(g_act * g_w).
struct Fp4Params {
    Params p;
    const float *g_act, *g_w;      // [1] or null (1)
    int direct;                    // pair kernel: the output takes plain stores (rows not 16-byte strided)
};

// Instruction descriptor of kind::mxf4 / mxf4nvf4, dense, K-major, E2M1 x E2M1
// -> f32: B scale id at bit 4, the element formats (1: E2M1) at 7 and 10,
// N / 8 at 17, the scale format (1: E8M0, 0: E4M3) at 23, M / 128 at 27, A
// scale id at 29.  A scale id is the byte of a TMEM word at which this
// instruction's scales start.
template <int FMT>
__host__ __device__ constexpr uint32_t idesc_fp4(int m, int n, int id)
{
    return (static_cast<uint32_t>(id) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           ((FMT == FMT_MX ? 1u : 0u) << 23) | (static_cast<uint32_t>(m >> 7) << 27) |
           (static_cast<uint32_t>(id) << 29);
}

// Shared-memory descriptor of one scale tile: 32 rows of 16 bytes without
// swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc_scales(saddr)) : "memory");
}

// This lane's 16 bytes of a scale tile in shared memory.
__device__ __forceinline__ void load_scale_words(uint32_t *d, uint32_t a)
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(a) : "memory");
}

// N words (8 or 16) of this thread's TMEM lane from registers.
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t *r)
{
    if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                     "%13, %14, %15, %16};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                     "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                     : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_st_all(uint32_t taddr, const uint32_t *r)
{
    static_assert(N % 8 == 0, "whole stores");
    constexpr int S = N % 16 == 0 ? 16 : 8;
#pragma unroll
    for (int i = 0; i < N; i += S) tmem_st<S>(taddr + i, r + i);
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int FMT, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate)
{
#define SQ_MMA_FP4(CGS, KINDS)                                                                         \
    asm volatile("{\n\t.reg .pred p;\n\t"                                                              \
                 "setp.ne.b32 p, %4, 0;\n\t"                                                           \
                 "tcgen05.mma.cta_group::" CGS "." KINDS " [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(d), \
                 "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)                      \
                 : "memory")
    if constexpr (FMT == FMT_MX && CG == 1) SQ_MMA_FP4("1", "kind::mxf4.block_scale.scale_vec::2X");
    else if constexpr (FMT == FMT_MX) SQ_MMA_FP4("2", "kind::mxf4.block_scale.scale_vec::2X");
    else if constexpr (CG == 1) SQ_MMA_FP4("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
    else SQ_MMA_FP4("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
#undef SQ_MMA_FP4
}

// fl(g_act * g_w), absent factors 1
__device__ __forceinline__ float out_factor(const Fp4Params &fp)
{
    return __fmul_rn(fp.g_act != nullptr ? __ldg(fp.g_act) : 1.0f, fp.g_w != nullptr ? __ldg(fp.g_w) : 1.0f);
}

// ---------------------------------------------------------------------------
// Few tiles: A = weights [N, K], B = activations [M, K] in tiles of BN tokens
// (more than one for BN = 64 and 128 only); a TMEM lane is an output channel, a column
// a token.  A cluster of CS
// CTAs shares a weight tile's K range; two CTAs fit an SM.  The partial sums
// are reduced by the whole cluster: groups of four tokens are dealt out to the
// CTAs in turn, and each is sent the others' sums of its own (st.async into its
// stages, which its MMAs have finished with, counted on its barrier).  Sums are
// taken in the order own, then by rank.  (Scales by tcgen05.st as in the pair
// kernel were 0.2-0.6 us slower: these products wait for the weights.)
// ---------------------------------------------------------------------------
template <int BN, int FMT>
struct SwapCfg {
    using Sf = SfT<FMT>;
    static constexpr int A_BYTES = BM * BKB, B_BYTES = BN * BKB;
    static constexpr int SF_BYTES = Sf::TILES * SF_TILE;           // of one operand's 128 rows
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + 2 * SF_BYTES;
    static constexpr int FIXED_BYTES = 1024 + 256;
    static constexpr int MAX_STAGES = 10;
    static constexpr int SF_COLS = Sf::TILES * 4;
    static constexpr int TMEM_COLS = gemm::pow2_at_least(BN + 2 * SF_COLS, 32);
    // stages and bytes of shared memory with one or two CTAs an SM
    static constexpr int stages(int per_sm)
    {
        const int n = ((per_sm == 1 ? 224 : 112) * 1024 - FIXED_BYTES) / STAGE_BYTES;
        return n < MAX_STAGES ? n : MAX_STAGES;
    }
    static constexpr int smem_bytes(int per_sm) { return FIXED_BYTES + stages(per_sm) * STAGE_BYTES; }
    static_assert(STAGE_BYTES % 1024 == 0, "stage must keep 1024-byte alignment");
    static_assert((2 * MAX_STAGES + 4) * 8 + 16 <= 256, "barrier area");
    static_assert(TMEM_COLS <= 256, "accumulators and scales of two CTAs must fit TMEM");
};

// N consecutive columns (4 or 16) of this thread's TMEM lane
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N])
{
    if constexpr (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr)
                     : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                     "%14, %15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(taddr)
                     : "memory");
}

template <int BN, int CS, int FMT>
__global__ void __launch_bounds__(NUM_THREADS, 2)
    k_fp4_swap(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
               const __grid_constant__ CUtensorMap map_ws, const __grid_constant__ CUtensorMap map_xs,
               const Fp4Params fp)
{
    using C = SwapCfg<BN, FMT>;
    using Sf = SfT<FMT>;
    // A scale address has to lie on an even TMEM column (64 rows): narrower
    // tiles than 64 tokens come alone (M <= BN).
    static_assert((CS - 1) * ((BN / 4 + CS - 1) / CS) * 2048 <= C::stages(2) * C::STAGE_BYTES, "partial sums must fit the stages");
    const Params &p = fp.p;
    const int S = p.ring;                                  // stages

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S * C::STAGE_BYTES);
    const uint32_t bar0 = ptx::smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    const uint32_t tfull_bar = bar0 + 8u * (2 * S);
    const uint32_t done_bar = bar0 + 8u * (2 * S + 1);
    const uint32_t go_bar = bar0 + 8u * (2 * S + 2);      // every CTA of the cluster is done with its stages
    const uint32_t part_bar = bar0 + 8u * (2 * S + 3);    // the others' partial sums have arrived
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const uint32_t sbase = ptx::smem_addr(smem);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = CS > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
    // token tiles of one weight tile's clusters are tiles_r clusters apart
    const int cluster = static_cast<int>(blockIdx.x) / CS;
    const int tc = cluster / p.tiles_r, tile = cluster - tc * p.tiles_r;
    const int tokens = min(BN, p.M - tc * BN);             // of this tile
    const int groups = (tokens + 3) >> 2;                  // of four tokens
    auto owned = [&](int r) { return (groups - r + CS - 1) / CS; };      // groups r, r + CS, ...
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        ptx::mbar_init(tfull_bar, 1);
        ptx::mbar_init(done_bar, 1);
        if constexpr (CS > 1) {
            ptx::mbar_init(go_bar, CS);
            ptx::mbar_init(part_bar, 1);
        }
        *abort_flag = 0;
        ptx::fence_barrier_init();
        if constexpr (CS > 1) ptx::mbar_arrive_expect_tx(part_bar, static_cast<uint32_t>((CS - 1) * owned(rank) * 2048));
    }
    if (warp == 0 && lane == 0) {
        ptx::tma_prefetch_desc(&map_w);
        ptx::tma_prefetch_desc(&map_x);
        ptx::tma_prefetch_desc(&map_ws);
        ptx::tma_prefetch_desc(&map_xs);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    if constexpr (CS > 1) ptx::cluster_sync();   // every CTA's barriers exist before any remote arrive
    ptx::tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint64_t tmo = p.timeout_ns;
    // this CTA's share of its tile's K blocks
    const int kb_begin = static_cast<int>(static_cast<int64_t>(rank) * p.num_kb / CS);
    const int kb_end = static_cast<int>(static_cast<int64_t>(rank + 1) * p.num_kb / CS);
    pdl_wait();                        // operands and scales come from the previous kernels

    // producer and MMA issuer walk their loops as whole warps (see k_fp4_pair)
    const bool issuer = ptx::elect_one();
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned code) {
        return __all_sync(0xffffffffu, ptx::wait_bounded(bar, parity, tmo, abort_flag, code));
    };
    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        for (int kb = kb_begin; kb < kb_end; ++kb) {
            if (!wait(empty_bar(stage), phase ^ 1u, ERR_PRODUCER)) break;
            const bool withhold = p.inject == 1 && blockIdx.x == 0 && issued == 0;
            if (issuer && !withhold) {
                const uint32_t fb = full_bar(stage);
                ptx::mbar_arrive_expect_tx(fb, C::STAGE_BYTES);
                const uint32_t sa = sbase + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                const uint32_t ssa = sb + C::B_BYTES, ssb = ssa + C::SF_BYTES;
                ptx::tma_load_2d(sa, &map_w, fb, kb * BKB, tile * BM);
                ptx::tma_load_3d(ssa, &map_ws, fb, 0, kb * Sf::TILES, tile);
                ptx::tma_load_2d(sb, &map_x, fb, kb * BKB, tc * BN);
                ptx::tma_load_3d(ssb, &map_xs, fb, 0, kb * Sf::TILES, tc * BN / 128);
            }
            __syncwarp();
            ++issued;
            if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        // drain: every issued load lands before the CTA exits
        const int n_wait = issued < S ? issued : S;
        for (int i = 0; i < n_wait; ++i) {
            int s = stage - 1 - i;
            uint32_t ph = phase;
            if (s < 0) { s += S; ph ^= 1u; }
            volatile int no_abort = 0;
            ptx::wait_bounded(full_bar(s), ph, tmo, &no_abort, ERR_DRAIN);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        // a tile's tokens start in the middle of a scale tile: 32 rows a TMEM column
        const uint32_t sfa0 = tmem_base + BN, sfb0 = sfa0 + C::SF_COLS, shift = (tc * BN) % 128 / 32;
        for (int kb = kb_begin; kb < kb_end; ++kb) {
            ok = wait(full_bar(stage), phase, ERR_MMA + 1);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t sa = sbase + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
            const uint32_t ssa = sb + C::B_BYTES, ssb = ssa + C::SF_BYTES;
            if (issuer) {
#pragma unroll
                for (int i = 0; i < Sf::TILES; ++i) {
                    copy_scales(sfa0 + 4 * i, ssa + i * SF_TILE);
                    copy_scales(sfb0 + 4 * i, ssb + i * SF_TILE);
                }
                const uint64_t ad = ptx::sdesc_kmajor_sw128(sa), bd = ptx::sdesc_kmajor_sw128(sb);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = k / Sf::MMAS;
                    mma_fp4<FMT, 1>(tmem_base, ad + 2 * k, bd + 2 * k, idesc_fp4<FMT>(128, BN, (k % Sf::MMAS) * 2),
                                    sfa0 + 4 * t, sfb0 + 4 * t + shift, (kb > kb_begin || k > 0) ? 1u : 0u);
                }
                ptx::tc_commit(empty_bar(stage));
            }
            __syncwarp();
            if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        if (issuer) {
            if (ok) ptx::tc_commit(tfull_bar);
            // drain: all issued MMAs complete before TMEM is released
            ptx::tc_commit(done_bar);
            volatile int no_abort = 0;
            ptx::wait_bounded(done_bar, 0u, tmo, &no_abort, ERR_DRAIN + 1);
        }
    } else {
        // ------------------------------------------------ epilogue (warps 2..5)
        const int q = warp & 3, r = q * 32 + lane, n = tile * BM + r;
        const float factor = out_factor(fp);
        // without a bias -0.0: the multiply-add then is the rounded product, sign of zero included
        const float bn = p.bias != nullptr && n < p.N ? gemm::load_bias(p.bias, p.out_dt, n) : -0.0f;
        const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        bool ok = wait(tfull_bar, 0u, ERR_EPI);
        ptx::tc_fence_after();
        if constexpr (CS > 1) {
            // [sender][owned group][row][4 tokens] in the owner's stages
            if (ok && q == 2 && lane < CS) ptx::mbar_arrive_plain(ptx::map_to_rank(go_bar, lane));
            ok = ok && wait(go_bar, 0u, ERR_EPI + 4);
            if (ok) {
#pragma unroll 1
                for (int c = 0; c < groups; c += 4) {
                    uint32_t v[16];
                    tmem_ld<16>(tbase + c * 4, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int g = c + i, owner = g % CS;
                        if (g < groups && owner != rank) {
                            const int slot = rank < owner ? rank : rank - 1;
                            const uint32_t off = static_cast<uint32_t>(((slot * owned(owner) + g / CS) * BM + r) * 16);
                            ptx::st_async_v4(ptx::map_to_rank(sbase + off, owner), ptx::map_to_rank(part_bar, owner), v[4 * i],
                                             v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    }
                }
                ok = __all_sync(0xffffffffu, ptx::wait_bounded_cluster(part_bar, 0u, tmo, abort_flag, ERR_EPI + 3));
            }
        }
        // this CTA's groups, four a step, with the output's type known at compile time
        const int mine = owned(rank);
        auto emit = [&](auto dt) {
            constexpr int DT = decltype(dt)::value;
            constexpr int SZ = dtype_size(DT);
            uint8_t *out = static_cast<uint8_t *>(p.out) + ((static_cast<int64_t>(tc) * BN + rank * 4) * p.N + n) * SZ;
            const int64_t token = static_cast<int64_t>(p.N) * SZ;
#pragma unroll 1
            for (int j = 0; j < mine; j += 4) {
                uint32_t v[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld<4>(tbase + (min(j + i, mine - 1) * CS + rank) * 4, v[i]);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (j + i < mine) {
                        float acc[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t) acc[t] = __uint_as_float(v[i][t]);
#pragma unroll
                        for (int s = 0; s < CS - 1; ++s) {
                            float4 o;
                            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                         : "=f"(o.x), "=f"(o.y), "=f"(o.z), "=f"(o.w)
                                         : "r"(sbase + static_cast<uint32_t>(((s * mine + j + i) * BM + r) * 16))
                                         : "memory");
                            acc[0] += o.x;
                            acc[1] += o.y;
                            acc[2] += o.z;
                            acc[3] += o.w;
                        }
                        const int left = n < p.N ? tokens - ((j + i) * CS + rank) * 4 : 0;
                        if (left >= 4) {
#pragma unroll
                            for (int t = 0; t < 4; ++t) gemm::store_out(out + t * token, DT, 0, __fmaf_rn(acc[t], factor, bn));
                        } else {
#pragma unroll
                            for (int t = 0; t < 3; ++t)
                                if (t < left) gemm::store_out(out + t * token, DT, 0, __fmaf_rn(acc[t], factor, bn));
                        }
                        out += 4 * CS * token;
                    }
                }
            }
        };
        if (ok) {
            if (p.out_dt == DT_BF16) emit(std::integral_constant<int, DT_BF16>());
            else if (p.out_dt == DT_F16) emit(std::integral_constant<int, DT_F16>());
            else emit(std::integral_constant<int, DT_F32>());
        }
        ptx::tc_fence_before();
    }

    __syncwarp();
    __syncthreads();
    if constexpr (CS > 1) ptx::cluster_meet();   // no CTA leaves while another may still write to its stages
    pdl_trigger();                     // every output of this CTA is written
    if (warp == 1) {
        // A CTA that gave up may have been sent partial sums that it did not
        // wait for: issued before the meeting, but asynchronous.  It stays
        // until they have landed (a store within the cluster takes ~1 us).
        if (CS > 1 && *abort_flag != 0) {
            for (int i = 0; i < 50; ++i) __nanosleep(1000);
        }
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// Large M: CTA pairs, 256 x BN tiles.  TMEM holds two accumulators and the
// scale columns of SF_BUFS stages.  256-wide tiles leave no room for two whole
// accumulators beside the scales: the second starts ACC_STRIDE < BN columns
// behind the first and shares OVERLAP columns with it.  The epilogue drains the
// shared columns first, and the next tile's MMAs start once they are free, so
// the rest of the epilogue still overlaps them.
// ---------------------------------------------------------------------------
constexpr int PAIR_THREADS = 352;      // gemm.cuh's six warps, four scale warps, the scale producer

constexpr int SF_BUFS_MX = 4, SF_BUFS_NV = 2;
constexpr int SF_SLOTS_MIN = 4;

template <int BN, int FMT>
struct Pair4Cfg {
    using Sf = SfT<FMT>;
    static constexpr int A_BYTES = BM * BKB, B_BYTES = (BN / 2) * BKB;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int NB = (BN % 128) == 0 ? BN / 128 : BN / 128 + 1;     // row tiles of B's scales
    static constexpr int SFA_BYTES = Sf::TILES * SF_TILE, SFB_BYTES = NB * SFA_BYTES;
    static constexpr int SF_BYTES = SFA_BYTES + SFB_BYTES;                   // a scale slot
    static constexpr int STG_TOTAL = 4 * 2 * STG_BYTES;     // two buffers a warp, 32 rows x 128 bytes each
    static constexpr int COLS_BYTES = 2 * 256 * 4;          // the tile's bias, two tiles
    static constexpr int FIXED_BYTES = 1024 + STG_TOTAL + COLS_BYTES + 512;
    static constexpr int ROOM = 227 * 1024 - FIXED_BYTES;
    static constexpr int STAGES_RAW = (ROOM - SF_SLOTS_MIN * SF_BYTES) / STAGE_BYTES;
    static constexpr int STAGES = STAGES_RAW > 10 ? 10 : STAGES_RAW;
    static constexpr int SLOTS_RAW = (ROOM - STAGES * STAGE_BYTES) / SF_BYTES;
    static constexpr int SLOTS = SLOTS_RAW > 8 ? 8 : SLOTS_RAW;
    static constexpr int SMEM_BYTES = FIXED_BYTES + STAGES * STAGE_BYTES + SLOTS * SF_BYTES;
    static constexpr int SFA_COLS = Sf::TILES * 4, SFB_COLS = NB * SFA_COLS;
    static constexpr int SF_COLS = SFA_COLS + SFB_COLS;     // of one stage
    static constexpr int SF_BUFS = FMT == FMT_MX ? SF_BUFS_MX : SF_BUFS_NV;
    static constexpr int ACC_ROOM = (512 - SF_BUFS * SF_COLS - BN) / 32 * 32;
    static constexpr int ACC_STRIDE = ACC_ROOM < BN ? ACC_ROOM : BN;
    static constexpr int OVERLAP = BN - ACC_STRIDE;         // a multiple of 32
    static constexpr int SF_COL0 = ACC_STRIDE + BN;
    static constexpr int TMEM_COLS = gemm::pow2_at_least(SF_COL0 + SF_BUFS * SF_COLS, 32);
    static_assert(STAGE_BYTES % 1024 == 0 && SF_BYTES % 128 == 0, "alignment of swizzled tiles and of scale slots");
    static_assert(BN % 64 == 0 && BN >= 128 && BN <= 256, "pair MMA N");
    static_assert(TMEM_COLS <= 512 && ACC_STRIDE > 0, "accumulators and scales must fit TMEM");
    static_assert(SF_BUFS <= STAGES && SLOTS >= 2, "a scale buffer's MMAs are told done by their stage's barrier");
    static_assert((2 * STAGES + 6 + 2 * SLOTS + SF_BUFS) * 8 + 16 <= 512, "barrier area");
};

// Factor and bias of 32 accumulator columns, in place.
template <bool BIAS>
__device__ __forceinline__ void apply_factor(uint32_t (&r)[32], float factor, const float *bias_tile)
{
    if constexpr (BIAS) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 b4 = *reinterpret_cast<const float4 *>(bias_tile + i);    // broadcast
            const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int t = 0; t < 4; ++t) r[i + t] = __float_as_uint(__fmaf_rn(__uint_as_float(r[i + t]), factor, bb[t]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__fmul_rn(__uint_as_float(r[i]), factor));
    }
}

template <int DT>
__device__ __forceinline__ uint32_t pack_out(uint32_t a, uint32_t b)
{
    if constexpr (DT == DT_F16) {
        const __half2 h = __floats2half2_rn(__uint_as_float(a), __uint_as_float(b));
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// The accumulator at tbase (128 lanes x BN columns): factor, bias, rounding,
// store, 64 columns a step; drained(i) is called when step i's columns are in
// registers.  Outputs leave through a staging buffer of 32 rows x 128 bytes in
// the output map's swizzle: 32 columns of 32-bit outputs, 64 of 16-bit ones.
// The type and the bias are compile-time here: with run-time branches in every
// chunk the epilogue took 3.4 us a 256-wide tile.
template <int BN, int DT, bool BIAS, typename Drained>
__device__ __forceinline__ void epilogue_pair(const Fp4Params &fp, const CUtensorMap *omap, uint32_t tbase, int ncol0,
                                              int mrow0, int lane, uint32_t stg, int &nstore, float factor,
                                              const float *bias_tile, bool reversed, Drained drained)
{
    const Params &p = fp.p;
#pragma unroll 1
    for (int i = 0; i < BN / 64; ++i) {
        const int c = (reversed ? BN / 64 - 1 - i : i) * 64;
        uint32_t r[2][32];
        ptx::tmem_ld32(tbase + c, r[0]);
        ptx::tmem_ld32(tbase + c + 32, r[1]);
        ptx::tmem_ld_wait();
        drained(i);
        const int n0 = ncol0 + c;
        if (n0 >= p.N) continue;
        apply_factor<BIAS>(r[0], factor, bias_tile + c);
        apply_factor<BIAS>(r[1], factor, bias_tile + c + 32);
        if (fp.direct) {
            // rows that no tensor map can describe: transposed through the
            // staging buffer (rotated rows: no bank conflicts), a row a step
            const int rows = min(32, p.M - mrow0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(stg + lane * 128 + ((j + lane) & 31) * 4), "r"(r[h][j]) : "memory");
                __syncwarp();
                const int n = n0 + 32 * h + lane;
                if (n < p.N) {
#pragma unroll 4
                    for (int j = 0; j < rows; ++j) {
                        float t;
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(t) : "r"(stg + j * 128 + ((j + lane) & 31) * 4) : "memory");
                        gemm::store_out(p.out, DT, static_cast<int64_t>(mrow0 + j) * p.N + n, t);
                    }
                }
                __syncwarp();
            }
            continue;
        }
        constexpr int STORES = DT == DT_F32 ? 2 : 1;
#pragma unroll
        for (int h = 0; h < STORES; ++h) {
            // a buffer is rewritten only once the store issued from it two
            // stores ago has finished reading shared memory
            if (lane == 0) ptx::bulk_wait_read_1();
            __syncwarp();
            const uint32_t buf = stg + static_cast<uint32_t>(nstore & 1) * STG_BYTES;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if constexpr (DT == DT_F32) w[t] = r[h][4 * k + t];
                    else w[t] = pack_out<DT>(r[k / 4][8 * (k & 3) + 2 * t], r[k / 4][8 * (k & 3) + 2 * t + 1]);
                }
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((k ^ (lane & 7)) << 4)),
                             "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                             : "memory");
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (DT != DT_F32 || n0 + 32 * h < p.N) ptx::tma_store_2d(omap, buf, n0 + 32 * h, mrow0);
                ptx::bulk_commit();
            }
            ++nstore;
        }
    }
}

template <int BN, int FMT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PAIR_THREADS, 1)
    k_fp4_pair(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_as, const __grid_constant__ CUtensorMap map_bs,
               const __grid_constant__ CUtensorMap map_o, const Fp4Params fp)
{
    using C = Pair4Cfg<BN, FMT>;
    using Sf = SfT<FMT>;
    constexpr int S = C::STAGES;
    const Params &p = fp.p;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *after = smem + S * C::STAGE_BYTES + C::SLOTS * C::SF_BYTES;       // behind the rings
    uint64_t *bars = reinterpret_cast<uint64_t *>(after + C::STG_TOTAL + C::COLS_BYTES);
    const uint32_t bar0 = ptx::smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * S + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
    const uint32_t done_bar = bar0 + 8u * (2 * S + 4);
    const uint32_t shared_bar = bar0 + 8u * (2 * S + 5);       // the shared accumulator columns are drained
    auto sf_full_bar = [&](int s) { return bar0 + 8u * (2 * S + 6 + s); };           // a slot of this CTA's scales is loaded
    auto sf_empty_bar = [&](int s) { return bar0 + 8u * (2 * S + 6 + C::SLOTS + s); };
    auto sf_ready_bar = [&](int b) { return bar0 + 8u * (2 * S + 6 + 2 * C::SLOTS + b); };   // both CTAs' scales are in TMEM
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S + 6 + 2 * C::SLOTS + C::SF_BUFS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *ok_flag = reinterpret_cast<volatile int *>(tmem_slot + 2);     // [2]
    const uint32_t sbase = ptx::smem_addr(smem);
    const uint32_t sf_base = sbase + S * C::STAGE_BYTES;
    const uint32_t stg_base = ptx::smem_addr(after);
    float *cols = reinterpret_cast<float *>(after + C::STG_TOTAL);   // [2][256] bias

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = (rank == 0);
    const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int s = 0; s < C::SLOTS; ++s) {
            ptx::mbar_init(sf_full_bar(s), 1);
            ptx::mbar_init(sf_empty_bar(s), 4);
        }
        for (int b = 0; b < C::SF_BUFS; ++b) ptx::mbar_init(sf_ready_bar(b), 8);
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(tfull_bar(b), 1);
            ptx::mbar_init(tempty_bar(b), 8);
        }
        ptx::mbar_init(done_bar, 1);
        ptx::mbar_init(shared_bar, 8);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::tma_prefetch_desc(&map_a);
        ptx::tma_prefetch_desc(&map_b);
        ptx::tma_prefetch_desc(&map_as);
        ptx::tma_prefetch_desc(&map_bs);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), C::TMEM_COLS);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();               // both CTAs' barriers exist before any remote use
    ptx::tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint64_t tmo = p.timeout_ns;
    pdl_wait();                        // operands and scales come from the previous kernels

    // The producers and the MMA issuer walk their loops as whole warps, so that
    // addresses and descriptors are warp-uniform (uniform registers feed these
    // instructions); one elected lane issues.  With one lane walking alone a
    // K block took 0.34 us however narrow the tile, against 0.27 us.
    const bool issuer = ptx::elect_one();
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned code) {
        return __all_sync(0xffffffffu, ptx::wait_bounded(bar, parity, tmo, abort_flag, code));
    };
    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = cluster; u < p.num_units && ok; u += nclusters) {
            int tr, tc;
            gemm::decode_unit(p, u, tr, tc);
            const int ya = (2 * tr + static_cast<int>(rank)) * BM;
            const int yb = tc * BN + static_cast<int>(rank) * (BN / 2);
            for (int kb = 0; kb < p.num_kb; ++kb) {
                ok = wait(empty_bar(stage), phase ^ 1u, ERR_PRODUCER);
                if (!ok) break;
                const bool withhold = p.inject == 1 && blockIdx.x == 0 && issued == 0;
                if (issuer && !withhold) {
                    if (leader) ptx::mbar_arrive_expect_tx(full_bar(stage), 2 * C::STAGE_BYTES);
                    const uint32_t fb = ptx::map_to_rank(full_bar(stage), 0);
                    const uint32_t sa = sbase + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                    ptx::tma_load_2d_pair(sa, &map_a, fb, kb * BKB, ya);
                    ptx::tma_load_2d_pair(sb, &map_b, fb, kb * BKB, yb);
                }
                __syncwarp();
                ++issued;
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
        }
        // drain: the leader's full barriers count both CTAs' bytes
        if (leader) {
            const int n_wait = issued < S ? issued : S;
            for (int i = 0; i < n_wait; ++i) {
                int s = stage - 1 - i;
                uint32_t ph = phase;
                if (s < 0) { s += S; ph ^= 1u; }
                volatile int no_abort = 0;
                ptx::wait_bounded(full_bar(s), ph, tmo, &no_abort, ERR_DRAIN);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader only)
        if (leader) {
            int stage = 0, local = 0, buf = 0;
            uint32_t phase = 0, bphase = 0;
            for (int u = cluster; u < p.num_units; u += nclusters, ++local) {
                const int b = local & 1;
                const uint32_t use = static_cast<uint32_t>(local >> 1) & 1u;
                if (!wait(tempty_bar(b), use ^ 1u, ERR_MMA)) break;
                if (C::OVERLAP > 0 && local > 0 && !wait(shared_bar, static_cast<uint32_t>(local - 1) & 1u, ERR_MMA + 2)) break;
                ptx::tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(b * C::ACC_STRIDE);
                int tr, tc;
                gemm::decode_unit(p, u, tr, tc);
                // a tile that starts in the middle of a row tile of scales
                // starts 2 columns (64 rows) into it
                const uint32_t shift = (BN % 128) != 0 ? static_cast<uint32_t>((tc * BN) % 128 / 32) : 0u;
                bool ok = true;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    ok = wait(sf_ready_bar(buf), bphase, ERR_MMA + 3) && wait(full_bar(stage), phase, ERR_MMA + 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t sa = sbase + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                    const uint32_t sfa0 = tmem_base + C::SF_COL0 + buf * C::SF_COLS, sfb0 = sfa0 + C::SFA_COLS + shift;
                    if (issuer) {
                        const uint64_t ad = ptx::sdesc_kmajor_sw128(sa), bd = ptx::sdesc_kmajor_sw128(sb);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int t = k / Sf::MMAS;
                            mma_fp4<FMT, 2>(d, ad + 2 * k, bd + 2 * k, idesc_fp4<FMT>(256, BN, (k % Sf::MMAS) * 2),
                                            sfa0 + 4 * t, sfb0 + 4 * C::NB * t, (kb > 0 || k > 0) ? 1u : 0u);
                        }
                        ptx::tc_commit_pair_mc(empty_bar(stage), 0x3);
                    }
                    __syncwarp();
                    if (++stage == S) { stage = 0; phase ^= 1u; }
                    if (++buf == C::SF_BUFS) { buf = 0; bphase ^= 1u; }
                }
                if (!ok) break;
                if (issuer) ptx::tc_commit_pair_mc(tfull_bar(b), 0x3);
                __syncwarp();
            }
            if (issuer) {
                ptx::tc_commit_pair(done_bar);
                volatile int no_abort = 0;
                ptx::wait_bounded(done_bar, 0u, tmo, &no_abort, ERR_DRAIN + 1);
            }
        }
    } else if (warp == 10) {
        // ------------------------------------------------ scale producer (both CTAs)
        int slot = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = cluster; u < p.num_units && ok; u += nclusters) {
            int tr, tc;
            gemm::decode_unit(p, u, tr, tc);
            const int ta = 2 * tr + static_cast<int>(rank);                  // 128-row tile of A
            for (int kb = 0; kb < p.num_kb; ++kb) {
                ok = wait(sf_empty_bar(slot), phase ^ 1u, ERR_PRODUCER + 1);
                if (!ok) break;
                if (issuer) {
                    const uint32_t fb = sf_full_bar(slot);
                    const uint32_t ssa = sf_base + slot * C::SF_BYTES;
                    ptx::mbar_arrive_expect_tx(fb, C::SF_BYTES);
                    ptx::tma_load_3d(ssa, &map_as, fb, 0, kb * Sf::TILES, ta);
                    ptx::tma_load_3d(ssa + C::SFA_BYTES, &map_bs, fb, 0, kb * Sf::TILES, tc * BN / 128);
                }
                __syncwarp();
                ++issued;
                if (++slot == C::SLOTS) { slot = 0; phase ^= 1u; }
            }
        }
        const int n_wait = issued < C::SLOTS ? issued : C::SLOTS;
        for (int i = 0; i < n_wait; ++i) {
            int s = slot - 1 - i;
            uint32_t ph = phase;
            if (s < 0) { s += C::SLOTS; ph ^= 1u; }
            volatile int no_abort = 0;
            ptx::wait_bounded(sf_full_bar(s), ph, tmo, &no_abort, ERR_DRAIN + 2);
        }
    } else if (warp >= 6) {
        // ------------------------------------------------ scales (warps 6..9, both CTAs)
        // TMEM lane l of every quarter holds rows l, 32 + l, 64 + l, 96 + l of
        // a scale tile: the 16 bytes at 16 * l.  Written from registers while
        // the MMAs of earlier stages run.
        const uint32_t tlane = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::SF_COL0;
        int slot = 0, buf = 0, old = 0, n = 0; // stage `old` was SF_BUFS stages before stage n
        uint32_t phase = 0, ophase = 0;
        bool ok = true;
        for (int u = cluster; u < p.num_units && ok; u += nclusters) {
            for (int kb = 0; kb < p.num_kb; ++kb) {
                ok = wait(sf_full_bar(slot), phase, ERR_MMA + 4);
                if (!ok) break;
                const uint32_t ssa = sf_base + slot * C::SF_BYTES + lane * 16, ssb = ssa + C::SFA_BYTES;
                uint32_t r[C::SF_COLS];
#pragma unroll
                for (int i = 0; i < Sf::TILES; ++i) {
                    load_scale_words(r + 4 * i, ssa + i * SF_TILE);
#pragma unroll
                    for (int t = 0; t < C::NB; ++t)
                        load_scale_words(r + C::SFA_COLS + 4 * (i * C::NB + t), ssb + (t * Sf::TILES + i) * SF_TILE);
                }
                if (n >= C::SF_BUFS) {         // the MMAs that read this buffer have completed
                    ok = wait(empty_bar(old), ophase, ERR_MMA + 5);
                    if (!ok) break;
                    if (++old == S) { old = 0; ophase ^= 1u; }
                    ptx::tc_fence_after();
                }
                ++n;
                tmem_st_all<C::SF_COLS>(tlane + buf * C::SF_COLS, r);
                tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive_plain(ptx::map_to_rank(sf_ready_bar(buf), 0));
                    ptx::mbar_arrive(sf_empty_bar(slot));        // every lane's words have arrived in registers
                }
                if (++slot == C::SLOTS) { slot = 0; phase ^= 1u; }
                if (++buf == C::SF_BUFS) buf = 0;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ epilogue (warps 2..5, both CTAs)
        const int q = warp & 3;
        const uint32_t stg = stg_base + static_cast<uint32_t>((warp - 2) * 2 * STG_BYTES);
        const float factor = out_factor(fp);
        int local = 0, nstore = 0;
        for (int u = cluster; u < p.num_units; u += nclusters, ++local) {
            int tr, tc;
            gemm::decode_unit(p, u, tr, tc);
            const int b = local & 1;
            const uint32_t use = static_cast<uint32_t>(local >> 1) & 1u;
            float *bias_tile = cols + b * 256;
            for (int t = threadIdx.x - 64; t < BN; t += 128) {
                const int n = tc * BN + t;
                bias_tile[t] = n < p.N ? gemm::load_bias(p.bias, p.out_dt, n) : 0.0f;
            }
            // one thread waits for the accumulator; the 128 epilogue threads
            // then take the same decision (no warp is left at a barrier alone)
            if (threadIdx.x == 64) ok_flag[b] = ptx::wait_bounded(tfull_bar(b), use, tmo, abort_flag, ERR_EPI) ? 1 : 0;
            ptx::named_bar_sync(1, 128);
            if (!ok_flag[b]) break;
            ptx::tc_fence_after();
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                   static_cast<uint32_t>(b * C::ACC_STRIDE);
            const int mrow0 = (2 * tr + static_cast<int>(rank)) * BM + q * 32;
            // the columns shared with the other accumulator first: the last
            // ones of the first accumulator, the first ones of the second
            auto drained = [&](int i) {
                const bool shared = C::OVERLAP > 0 && i == (C::OVERLAP - 1) / 64, last = i == BN / 64 - 1;
                if (shared || last) {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && shared) ptx::mbar_arrive_plain(ptx::map_to_rank(shared_bar, 0));
                    if (lane == 0 && last) ptx::mbar_arrive_plain(ptx::map_to_rank(tempty_bar(b), 0));
                }
            };
            auto run = [&](auto dt, auto bias) {
                epilogue_pair<BN, decltype(dt)::value, decltype(bias)::value>(fp, &map_o, tbase, tc * BN, mrow0, lane, stg,
                                                                              nstore, factor, bias_tile,
                                                                              C::OVERLAP > 0 && b == 0, drained);
            };
            auto by_dt = [&](auto bias) {
                if (p.out_dt == DT_BF16) run(std::integral_constant<int, DT_BF16>(), bias);
                else if (p.out_dt == DT_F16) run(std::integral_constant<int, DT_F16>(), bias);
                else run(std::integral_constant<int, DT_F32>(), bias);
            };
            if (p.bias != nullptr) by_dt(std::true_type());
            else by_dt(std::false_type());
        }
        if (lane == 0) ptx::bulk_wait_all();     // output stores complete before the CTA exits
        __syncwarp();
    }

    ptx::tc_fence_before();
    ptx::cluster_sync();               // no CTA leaves while its peer may still signal it
    pdl_trigger();                     // every output of this CTA is written (TMA stores waited for)
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace fp4
}  // namespace sq
