// fp4.cuh -- 4-bit microscaled floating point: quantisation of weights and
// activations to blocks of E2M1 codes, and back.
//
// Two formats (OCP Microscaling Formats specification v1.0 for MXFP4):
//   MXFP4: 32 codes share one E8M0 scale 2^(byte - 127)
//   NVFP4: 16 codes share one E4M3 scale, and the tensor one fp32 scale g
// E2M1 has the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 (codes 0..7, sign in
// bit 3); two codes a byte, the even column in the low nibble.
//
//   x'  = fl(x * recip(s_j)) (activations) or fl(w * s_j) (weights); x without s
//   m   = max |x'| over the block (columns past K count as 0)
//   MXFP4:  byte = max(exponent field of m - 2, 0), i.e. 2^(floor(log2 m) - 2)
//           held at 2^-127;  code = e2m1(x' * 2^(127 - byte))   (exact product)
//   NVFP4:  v = e4m3(fl(m * fl(recip(g) * fl(1/6))));  code = e2m1(fl(x' * recip(fl(v * g))))
//   value = fl(e2m1 * scale), scale = 2^(byte - 127) or fl(v * g)
// with recip(v) = min(fl(1/v), FLT_MAX) for v > 0, else 0.  A block that
// holds an infinity or a NaN gets the NaN scale (0xff, or 0x7f).
//
// Codes are row-major, 16 * ceil(K / 32) bytes a row (zero codes behind K).
// Scales are laid out for the tensor cores: tiles of 128 rows x 4 blocks (512
// bytes), tiles along K first; within a tile, row r's four bytes lie at
// 16 * (r % 32) + 4 * (r / 32).  That is the order in which tcgen05.cp's
// 32-lane x 128-bit copy brings a tile into tensor memory, so the product
// copies scales without touching them.  Bytes of blocks behind K are 0; rows
// behind the last one are not written.
#pragma once

#include "common.cuh"

namespace sq {
namespace fp4 {

enum Fmt : int { FMT_MX = 0, FMT_NV = 1 };

template <int FMT> struct FmtT {
    static constexpr int BLOCK = FMT == FMT_MX ? 32 : 16;
    static constexpr int TILE_K = 4 * BLOCK;               // columns of a scale tile
};

constexpr int SF_TILE = 512;                                // bytes of a scale tile

__host__ __device__ constexpr int64_t code_row_bytes(int64_t K) { return (K + 31) / 32 * 16; }
__host__ __device__ constexpr int64_t scale_tiles_k(int fmt, int64_t K)
{
    return ((K + 31) / 32 * (fmt == FMT_MX ? 1 : 2) + 3) / 4;
}

// byte offset of the 4-byte word of row r, tile kt along K
__device__ __forceinline__ int64_t scale_word(int64_t r, int64_t kt, int64_t ktiles)
{
    const int rr = static_cast<int>(r & 127);
    return ((r >> 7) * ktiles + kt) * SF_TILE + (rr & 31) * 16 + (rr >> 5) * 4;
}

__device__ __forceinline__ float recip_finite(float v)
{
    return v > 0.0f ? fminf(__frcp_rn(v), 3.4028234663852886e38f) : 0.0f;
}

// 8 values -> 8 codes (f[0] in bits 0..3), round to nearest even, beyond 6 saturated
__device__ __forceinline__ uint32_t e2m1x8(const float *f)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return r;
}

// 8 codes -> 8 values
__device__ __forceinline__ void e2m1x8_decode(uint32_t q, float *f)
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(q));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

// E4M3 code -> value (0x7f: NaN)
__device__ __forceinline__ float e4m3_value(uint32_t byte)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte & 0xffu)));
    return __half2float(__low2half(*reinterpret_cast<const __half2 *>(&h)));
}

// E8M0 scale 2^(byte - 127): byte 0 is the subnormal 2^-127, 255 is NaN
__device__ __forceinline__ float e8m0_value(uint32_t byte)
{
    return byte == 255u ? __uint_as_float(0x7fffffffu) : byte == 0u ? __uint_as_float(0x00400000u)
                                                                    : __uint_as_float(byte << 23);
}

// The scale byte of a block with absmax m (NaN and infinity come through m)
// and the factor its values are multiplied with before rounding.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(float m, float gc, float g, float &inv)
{
    if constexpr (FMT == FMT_MX) {
        const int e = static_cast<int>(__float_as_uint(m) >> 23);
        const uint32_t b = static_cast<uint32_t>(e > 2 ? e - 2 : 0);
        inv = __uint_as_float((254u - b) << 23);
        return e == 255 ? 255u : b;
    } else {
        const uint32_t b = e4m3x2_bits(__fmul_rn(m, gc), 0.0f) & 0xffu;
        inv = recip_finite(__fmul_rn(e4m3_value(b), g));
        return m < __uint_as_float(0x7f800000u) ? b : 0x7fu;
    }
}

// 16 elements as they lie in memory: VEC bytes a load (32 or 16; 0: one by one)
template <int DT> struct Raw16 { uint4 v[dtype_size(DT)]; };

__device__ __forceinline__ void load32(const void *p, uint4 &a, uint4 &b)
{
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
}

__device__ __forceinline__ void store32(void *p, const uint4 &a, const uint4 &b)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

// Elements [c, c + 16) of the row at `row`; those at n and behind are 0.
template <int DT, int VEC>
__device__ __forceinline__ void load16(const void *row, int64_t c, int64_t n, Raw16<DT> &r)
{
    constexpr int SZ = dtype_size(DT), NV = SZ;             // 16-byte pieces
    const uint8_t *p = static_cast<const uint8_t *>(row) + c * SZ;
    if (VEC == 32 && c + 16 <= n) {
#pragma unroll
        for (int i = 0; i < NV; i += 2) load32(p + 16 * i, r.v[i], r.v[i + 1]);
    } else if (VEC == 16 && c + 16 <= n) {
#pragma unroll
        for (int i = 0; i < NV; ++i) r.v[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    } else {
        uint32_t w[4 * NV];
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) {
            if constexpr (SZ == 4) {
                w[i] = c + i < n ? __ldg(reinterpret_cast<const uint32_t *>(p) + i) : 0u;
            } else {
                const uint32_t lo = c + 2 * i < n ? __ldg(reinterpret_cast<const uint16_t *>(p) + 2 * i) : 0u;
                const uint32_t hi = c + 2 * i + 1 < n ? __ldg(reinterpret_cast<const uint16_t *>(p) + 2 * i + 1) : 0u;
                w[i] = lo | (hi << 16);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) r.v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}

// load16 with the width known at run time only (the same for the whole warp)
template <int DT>
__device__ __forceinline__ void load16_rt(int vec, const void *row, int64_t c, int64_t n, Raw16<DT> &r)
{
    if (vec == 32) load16<DT, 32>(row, c, n, r);
    else if (vec == 16) load16<DT, 16>(row, c, n, r);
    else load16<DT, 0>(row, c, n, r);
}

template <int DT>
__device__ __forceinline__ void widen16(const Raw16<DT> &r, float (&f)[16])
{
    constexpr int EPV = VecT<DT>::EPV;
#pragma unroll
    for (int i = 0; i < dtype_size(DT); ++i) {
        float t[EPV];
        widen<DT>(r.v[i], t);
#pragma unroll
        for (int j = 0; j < EPV; ++j) f[i * EPV + j] = t[j];
    }
}

// 16 values of a row at column c, rounded to the output type; those at n and
// behind are not stored.  VEC as in load16.
template <int DT, int VEC>
__device__ __forceinline__ void store16(void *row, int64_t c, int64_t n, const float (&f)[16])
{
    constexpr int SZ = dtype_size(DT), NV = SZ;
    uint8_t *p = static_cast<uint8_t *>(row) + c * SZ;
    uint32_t w[4 * NV];
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) {
        if constexpr (DT == DT_F32) {
            w[i] = __float_as_uint(f[i]);
        } else if constexpr (DT == DT_F16) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    auto piece = [&](int i) { return make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]); };
    if (VEC == 32 && c + 16 <= n) {
#pragma unroll
        for (int i = 0; i < NV; i += 2) store32(p + 16 * i, piece(i), piece(i + 1));
    } else if (VEC == 16 && c + 16 <= n) {
#pragma unroll
        for (int i = 0; i < NV; ++i) reinterpret_cast<uint4 *>(p)[i] = piece(i);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (c + i < n) {
                if constexpr (SZ == 4) reinterpret_cast<uint32_t *>(p)[i] = w[i];
                else reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ void store16_rt(int vec, void *row, int64_t c, int64_t n, const float (&f)[16])
{
    if (vec == 32) store16<DT, 32>(row, c, n, f);
    else if (vec == 16) store16<DT, 16>(row, c, n, f);
    else store16<DT, 0>(row, c, n, f);
}

// ---------------------------------------------------------------------------
// Quantisation.  A thread owns 16 columns (one NVFP4 block, half an MXFP4
// block) and walks a slab of rows, so that the columns' smoothing constants
// stay in registers.  A warp covers 512 columns of a row.
// ---------------------------------------------------------------------------
constexpr int QTX = 32, QTY = 8;

struct QuantArgs {
    const void *x;
    int64_t rows, K, ld;       // ld: elements between rows
    const float *s;            // [K] or null
    const float *g;            // [1] or null (1): NVFP4's tensor scale
    uint8_t *q;
    uint8_t *sf;
    int64_t slab;              // rows per block
    int weight;                // multiply with s_j instead of recip(s_j)
};

template <int DT, int VEC, int FMT>
__global__ void __launch_bounds__(QTX *QTY) k_fp4_quant(const QuantArgs a)
{
    constexpr int TILE_K = FmtT<FMT>::TILE_K, SZ = dtype_size(DT);
    constexpr int U = 2;                                    // rows in flight per thread
    const int lane = threadIdx.x;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * QTX + lane) * 16;
    const int64_t ktiles = scale_tiles_k(FMT, a.K), qld = code_row_bytes(a.K);
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * a.slab, r1 = min(r0 + a.slab, a.rows);
    pdl_wait();
    float cs[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float s = a.s != nullptr && c + i < a.K ? __ldg(a.s + c + i) : 1.0f;
        cs[i] = a.s == nullptr ? 1.0f : a.weight ? s : recip_finite(s);
    }
    float g = 1.0f, gc = 0.0f;
    if constexpr (FMT == FMT_NV) {
        if (a.g != nullptr) g = __ldg(a.g);
        gc = __fmul_rn(recip_finite(g), 1.0f / 6.0f);
    }
    for (int64_t r = r0 + threadIdx.y; r < r1; r += U * QTY) {
        Raw16<DT> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r + u * QTY < r1)
                load16<DT, VEC>(static_cast<const uint8_t *>(a.x) + (r + u * QTY) * a.ld * SZ, c, a.K, raw[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = r + u * QTY;
            if (row >= r1) break;                           // the same for the whole warp
            float f[16];
            widen16<DT>(raw[u], f);
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 t = __fmul2_rn(make_float2(f[i], f[i + 1]), make_float2(cs[i], cs[i + 1]));
                f[i] = t.x;
                f[i + 1] = t.y;
                m = max3_abs_nan(m, t.x, t.y);
            }
            if constexpr (FMT == FMT_MX) m = max3_abs_nan(m, __shfl_xor_sync(0xffffffffu, m, 1), 0.0f);
            float inv;
            const uint32_t b = block_scale<FMT>(m, gc, g, inv);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 t = __fmul2_rn(make_float2(f[i], f[i + 1]), make_float2(inv, inv));
                f[i] = t.x;
                f[i + 1] = t.y;
            }
            if (c < 2 * qld) *reinterpret_cast<uint2 *>(a.q + row * qld + (c >> 1)) = make_uint2(e2m1x8(f), e2m1x8(f + 8));
            // the four bytes of a scale tile's row, from the lanes that hold them
            constexpr int LB = FMT == FMT_MX ? 2 : 1;       // lanes per block
            uint32_t w = b << (8 * ((lane / LB) & 3));
            w |= __shfl_xor_sync(0xffffffffu, w, LB);
            w |= __shfl_xor_sync(0xffffffffu, w, 2 * LB);
            const int64_t kt = c / TILE_K;
            if (lane % (4 * LB) == 0 && kt < ktiles)
                *reinterpret_cast<uint32_t *>(a.sf + scale_word(row, kt, ktiles)) = w;
        }
    }
    __syncthreads();
    pdl_trigger();
}

// ---------------------------------------------------------------------------
// Values from codes: out[r, j] = RN_out(fl(e2m1(code) * scale)).
// ---------------------------------------------------------------------------
struct DequantArgs {
    const uint8_t *q, *sf;
    int64_t rows, K;
    const float *g;
    void *out;
    int64_t slab;
};

template <int DT, int VEC, int FMT>
__global__ void __launch_bounds__(QTX *QTY) k_fp4_dequant(const DequantArgs a)
{
    constexpr int TILE_K = FmtT<FMT>::TILE_K, SZ = dtype_size(DT);
    constexpr int U = 4;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * QTX + threadIdx.x) * 16;
    const int64_t ktiles = scale_tiles_k(FMT, a.K), qld = code_row_bytes(a.K);
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * a.slab, r1 = min(r0 + a.slab, a.rows);
    pdl_wait();
    const float g = (FMT == FMT_NV && a.g != nullptr) ? __ldg(a.g) : 1.0f;
    if (c < a.K) {
        const int64_t kt = c / TILE_K;
        const int byte = static_cast<int>(c % TILE_K) / FmtT<FMT>::BLOCK;
        for (int64_t r = r0 + threadIdx.y; r < r1; r += U * QTY) {
            uint2 q[U];
            uint32_t b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = r + u * QTY;
                if (row < r1) {
                    q[u] = __ldg(reinterpret_cast<const uint2 *>(a.q + row * qld + (c >> 1)));
                    b[u] = __ldg(a.sf + scale_word(row, kt, ktiles) + byte);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = r + u * QTY;
                if (row >= r1) break;
                const float sc = FMT == FMT_MX ? e8m0_value(b[u]) : __fmul_rn(e4m3_value(b[u]), g);
                float f[16];
                e2m1x8_decode(q[u].x, f);
                e2m1x8_decode(q[u].y, f + 8);
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = __fmul_rn(f[i], sc);
                store16<DT, VEC>(static_cast<uint8_t *>(a.out) + row * a.K * SZ, c, a.K, f);
            }
        }
    }
    __syncthreads();
    pdl_trigger();
}

// ---------------------------------------------------------------------------
// Smoothing factors with NVFP4's two tensor scales (one block):
//   s_j as sq_smooth_scales;  g_act = fl(max_j fl(act_max_j * recip(s_j)) / 2688),
//   g_w = fl(max_j fl(w_max_j * s_j) / 2688)      (2688 = 6 * 448)
// s comes from sq_smooth_scales' own kernel; this one reduces over it.
// ---------------------------------------------------------------------------
static __global__ void __launch_bounds__(1024) k_nvfp4_scales(const float *act_max, const float *w_max, int64_t K,
                                                              const float *s, float *g_act, float *g_w)
{
    __shared__ float red[32];
    pdl_wait();
    float ma = 0.0f, mw = 0.0f;
    for (int64_t j = threadIdx.x; j < K; j += 1024) {
        const float sj = __ldg(s + j);
        ma = fmaxf(ma, __fmul_rn(__ldg(act_max + j), recip_finite(sj)));
        mw = fmaxf(mw, __fmul_rn(__ldg(w_max + j), sj));
    }
    ma = block_max(ma, red);
    mw = block_max(mw, red);
    if (threadIdx.x == 0) {
        if (g_act != nullptr) *g_act = __fdiv_rn(ma, 2688.0f);
        if (g_w != nullptr) *g_w = __fdiv_rn(mw, 2688.0f);
    }
    __syncthreads();
    pdl_trigger();
}

}  // namespace fp4
}  // namespace sq
