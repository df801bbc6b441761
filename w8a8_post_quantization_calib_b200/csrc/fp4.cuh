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

// 16 elements as they lie in memory
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

// VEC bytes (16, 8 or 4) as 32-bit words
template <int VEC>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w)
{
    if constexpr (VEC == 16) {
        const uint4 t = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = t.x;
        w[1] = t.y;
        w[2] = t.z;
        w[3] = t.w;
    } else if constexpr (VEC == 8) {
        const uint2 t = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = t.x;
        w[1] = t.y;
    } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    }
}

template <int VEC>
__device__ __forceinline__ void store_words(uint8_t *p, const uint32_t *w)
{
    if constexpr (VEC == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(p) = w[0];
}

// Elements [c, c + 16) of the row at `row`; those at n and behind are 0.  VEC:
// bytes that the row's address and every 16-element piece of it allow (32, 16,
// 8, 4, or 0: single elements).
template <int DT, int VEC>
__device__ __forceinline__ void load16(const void *row, int64_t c, int64_t n, Raw16<DT> &r)
{
    constexpr int SZ = dtype_size(DT), NV = SZ;             // 16-byte pieces
    constexpr int PV = VEC == 32 ? 16 : VEC < SZ ? 0 : VEC; // bytes a piece of a chunk that ends inside
    const uint8_t *p = static_cast<const uint8_t *>(row) + c * SZ;
    if (VEC == 32 && c + 16 <= n) {
#pragma unroll
        for (int i = 0; i < NV; i += 2) load32(p + 16 * i, r.v[i], r.v[i + 1]);
        return;
    }
    uint32_t w[4 * NV];
    auto elements = [&](int i) {                            // word i from single elements
        if constexpr (SZ == 4) {
            w[i] = c + i < n ? __ldg(reinterpret_cast<const uint32_t *>(p) + i) : 0u;
        } else {
            const uint32_t lo = c + 2 * i < n ? __ldg(reinterpret_cast<const uint16_t *>(p) + 2 * i) : 0u;
            const uint32_t hi = c + 2 * i + 1 < n ? __ldg(reinterpret_cast<const uint16_t *>(p) + 2 * i + 1) : 0u;
            w[i] = lo | (hi << 16);
        }
    };
    if constexpr (PV >= 4) {
        constexpr int WP = PV / 4, EP = PV / SZ;
#pragma unroll
        for (int i = 0; i < 4 * NV; i += WP) {
            if (c + (i / WP + 1) * EP <= n) {
                load_words<PV>(p + 4 * i, w + i);
            } else {
#pragma unroll
                for (int j = 0; j < WP; ++j) elements(i + j);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) elements(i);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) r.v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// load16 with VEC 32 or 16 known at compile time, or a narrower width `vec`
// known at run time only (VEC = 0)
template <int DT, int VEC>
__device__ __forceinline__ void load16_rt(int vec, const void *row, int64_t c, int64_t n, Raw16<DT> &r)
{
    if constexpr (VEC != 0) load16<DT, VEC>(row, c, n, r);
    else if (vec == 8) load16<DT, 8>(row, c, n, r);
    else if (vec == 4) load16<DT, 4>(row, c, n, r);
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

// 16 values rounded to the output type, as words
template <int DT>
__device__ __forceinline__ void round16(const float (&f)[16], uint32_t (&w)[4 * dtype_size(DT)])
{
#pragma unroll
    for (int i = 0; i < 4 * dtype_size(DT); ++i) {
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
}

// 16 values of a row at column c, rounded to the output type; those at n and
// behind are not stored.  VEC as in load16.
template <int DT, int VEC>
__device__ __forceinline__ void store16(void *row, int64_t c, int64_t n, const float (&f)[16])
{
    constexpr int SZ = dtype_size(DT), NV = SZ;
    uint8_t *p = static_cast<uint8_t *>(row) + c * SZ;
    uint32_t w[4 * NV];
    round16<DT>(f, w);
    constexpr int PV = VEC == 32 ? 16 : VEC < SZ ? 0 : VEC;
    if (VEC == 32 && c + 16 <= n) {
#pragma unroll
        for (int i = 0; i < NV; i += 2)
            store32(p + 16 * i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]),
                    make_uint4(w[4 * i + 4], w[4 * i + 5], w[4 * i + 6], w[4 * i + 7]));
        return;
    }
    auto elements = [&](int i) {                            // word i as single elements
        if constexpr (SZ == 4) {
            if (c + i < n) reinterpret_cast<uint32_t *>(p)[i] = w[i];
        } else {
            if (c + 2 * i < n) reinterpret_cast<uint16_t *>(p)[2 * i] = static_cast<uint16_t>(w[i]);
            if (c + 2 * i + 1 < n) reinterpret_cast<uint16_t *>(p)[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
        }
    };
    if constexpr (PV >= 4) {
        constexpr int WP = PV / 4, EP = PV / SZ;
#pragma unroll
        for (int i = 0; i < 4 * NV; i += WP) {
            if (c + (i / WP + 1) * EP <= n) {
                store_words<PV>(p + 4 * i, w + i);
            } else {
#pragma unroll
                for (int j = 0; j < WP; ++j) elements(i + j);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) elements(i);
    }
}

template <int DT, int VEC>
__device__ __forceinline__ void store16_rt(int vec, void *row, int64_t c, int64_t n, const float (&f)[16])
{
    if constexpr (VEC != 0) store16<DT, VEC>(row, c, n, f);
    else if (vec == 8) store16<DT, 8>(row, c, n, f);
    else if (vec == 4) store16<DT, 4>(row, c, n, f);
    else store16<DT, 0>(row, c, n, f);
}

// Rows off 16 bytes.  A lane's 16 elements are loaded as the 16-byte vectors
// around them, one more than they take, and moved into place in registers; they
// are stored the other way round, with the end of the lane before in front.
// Loads may take bytes beside the row, but none outside [lo, hi), the tensor.

// words [0, N - 4) of the result start `bytes` (even, below 16) behind ext[0]
template <int N>
__device__ __forceinline__ void shift_words(uint32_t (&ext)[N], int bytes)
{
    if (bytes & 8) {
#pragma unroll
        for (int i = 0; i < N - 2; ++i) ext[i] = ext[i + 2];
    }
    if (bytes & 4) {
#pragma unroll
        for (int i = 0; i < N - 1; ++i) ext[i] = ext[i + 1];
    }
    if (bytes & 2) {
#pragma unroll
        for (int i = 0; i < N - 1; ++i) ext[i] = __funnelshift_r(ext[i], ext[i + 1], 16);
    }
}

template <int DT> struct Around16 { uint32_t w[4 * dtype_size(DT) + 4]; };

// The vectors around elements [c, c + 16) of the row; n: the row's elements.
template <int DT>
__device__ __forceinline__ void load_around(const uint8_t *row, int64_t c, int64_t n, const uint8_t *lo, const uint8_t *hi,
                                            Around16<DT> &r)
{
    constexpr int SZ = dtype_size(DT);
    const uint8_t *a = row + c * SZ;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(a) & 15);
    const uint8_t *p = a - off;
    const uint8_t *end = row + n * SZ;                      // vectors from here on hold nothing of the row
#pragma unroll
    for (int i = 0; i < SZ + 1; ++i, p += 16) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (p < end && (i < SZ || off != 0)) {
            if (p >= lo && p + 16 <= hi) {
                load_words<16>(p, w);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint8_t *e = p + 2 * j;
                    if (e >= lo && e < hi) w[j / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(e))) << (16 * (j & 1));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[4 * i + j] = w[j];
    }
}

// Elements [c, c + 16) of the row out of the vectors around them; 0 at n and behind.
template <int DT>
__device__ __forceinline__ void settle(const uint8_t *row, int64_t c, int64_t n, Around16<DT> &r, Raw16<DT> &out)
{
    constexpr int SZ = dtype_size(DT);
    shift_words(r.w, static_cast<int>(reinterpret_cast<uintptr_t>(row + c * SZ) & 15));
    if (c + 16 > n) {
#pragma unroll
        for (int i = 0; i < 4 * SZ; ++i) {
            if constexpr (SZ == 4) {
                if (c + i >= n) r.w[i] = 0u;
            } else {
                if (c + 2 * i >= n) r.w[i] = 0u;
                else if (c + 2 * i + 1 >= n) r.w[i] &= 0xffffu;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < SZ; ++i) out.v[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
}

// 512 values of a strip (16 a lane, `left` elements of the row from its start
// on) to any address of their type; the whole warp.
template <int DT>
__device__ __forceinline__ void store_strip(uint8_t *strip, int64_t left, int lane, const float (&f)[16])
{
    constexpr int SZ = dtype_size(DT), N = 4 * SZ;
    uint32_t w[N];
    round16<DT>(f, w);
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(strip) & 15);
    uint32_t ext[N + 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ext[i] = __shfl_up_sync(0xffffffffu, w[N - 4 + i], 1);
#pragma unroll
    for (int i = 0; i < N; ++i) ext[4 + i] = w[i];
    const int64_t bytes = left * SZ;
    if (off == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) ext[i] = w[i];
    } else {
        shift_words(ext, 16 - off);
    }
    // this lane's vectors: bytes o .. o + 15 of the strip
#pragma unroll
    for (int i = 0; i < SZ; ++i) {
        const int o = lane * 16 * SZ + 16 * i - off;
        if (o >= 0 && o + 16 <= bytes) {
            store_words<16>(strip + o, ext + 4 * i);
        } else {
#pragma unroll
            for (int j = 0; j < 16 / SZ; ++j) {
                const int e = o + j * SZ;
                if (e >= 0 && e < bytes) {
                    if constexpr (SZ == 4) *reinterpret_cast<uint32_t *>(strip + e) = ext[4 * i + j];
                    else *reinterpret_cast<uint16_t *>(strip + e) = static_cast<uint16_t>(ext[4 * i + j / 2] >> (16 * (j & 1)));
                }
            }
        }
    }
    // the strip's last `off` bytes lie behind the last lane's vectors
    if (lane == 31 && off != 0) {
#pragma unroll
        for (int j = 0; j < 16 / SZ; ++j) {
            const int e = 512 * SZ - 16 + j * SZ;
            if (e >= 512 * SZ - off && e < bytes) {
                if constexpr (SZ == 4) *reinterpret_cast<uint32_t *>(strip + e) = w[N - 4 + j];
                else *reinterpret_cast<uint16_t *>(strip + e) = static_cast<uint16_t>(w[N - 4 + j / 2] >> (16 * (j & 1)));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Rows and columns of a block of 32 x 8 threads: a warp covers 512 columns (16
// a lane: an NVFP4 block, half an MXFP4 block), a thread ROWS rows.  ROWS = 4: r,
// r + 32, r + 64, r + 96 of a 128-row scale tile, whose scale words lie in 16
// contiguous bytes; a unit is eight such r.  ROWS = 1 (a unit is eight rows) where
// that would leave SMs idle.  A block walks units, so that its columns'
// smoothing constants stay in registers.
// ---------------------------------------------------------------------------
constexpr int QTX = 32, QTY = 8;

template <int ROWS> __host__ __device__ constexpr int64_t quant_units(int64_t rows)
{
    if (ROWS == 1) return (rows + QTY - 1) / QTY;
    const int64_t last = rows & 127;                        // the last tile's units with at least one row
    return (rows >> 7) * 4 + (last >= 32 ? 4 : (last + QTY - 1) / QTY);
}
template <int ROWS> __device__ __forceinline__ int64_t unit_row(int64_t unit, int ty)
{
    return ROWS == 1 ? unit * QTY + ty : (unit >> 2) * 128 + (unit & 3) * QTY + ty;
}

// ---------------------------------------------------------------------------
// Quantisation.  Bound by memory: [16384, 8192] bf16 -> MXFP4 reads and writes
// 344 MB in 52.8 us, 6.5 TB/s, the measured copy rate; NVFP4 53.8 us.  What
// carries it: the factors' reciprocals taken once a block (with one set a
// thread a launch on 16 rows took 4.2 us, now 2.2), the next unit's loads issued
// before this one is computed (91 -> 53 us), and one pass of blocks over the SMs.
// ---------------------------------------------------------------------------
struct QuantArgs {
    const void *x;
    int64_t rows, K, ld;       // ld: elements between rows
    const float *s;            // [K] or null
    const float *g;            // [1] or null (1): NVFP4's tensor scale
    uint8_t *q;
    uint8_t *sf;
    int64_t units;
    int weight;                // multiply with s_j instead of recip(s_j)
};

// A row's 16 elements on their way: VEC 32 or 16, or (0) rows off 16 bytes.
template <int DT, int VEC> struct InFlight { Raw16<DT> v; };
template <int DT> struct InFlight<DT, 0> { Around16<DT> v; };

template <int DT, int VEC, int ROWS>
__device__ __forceinline__ void load_rows(const QuantArgs &a, int64_t r, int64_t c, InFlight<DT, VEC> (&raw)[ROWS])
{
    constexpr int SZ = dtype_size(DT);
    const uint8_t *x = static_cast<const uint8_t *>(a.x);
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        if (r + 32 * u >= a.rows) break;
        const uint8_t *row = x + (r + 32 * u) * a.ld * SZ;
        if constexpr (VEC != 0) load16<DT, VEC>(row, c, a.K, raw[u].v);
        else load_around<DT>(row, c, a.K, x, x + ((a.rows - 1) * a.ld + a.K) * SZ, raw[u].v);
    }
}

template <int DT, int VEC, int FMT, int ROWS>
__global__ void __launch_bounds__(QTX *QTY) k_fp4_quant(const QuantArgs a)
{
    constexpr int TILE_K = FmtT<FMT>::TILE_K;
    constexpr int LB = FMT == FMT_MX ? 2 : 1;               // lanes per block
    __shared__ float4 s_cs[4][QTX];                         // the strip's factors, [4 columns][lane]
    const int lane = threadIdx.x;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * QTX + lane) * 16;
    const int64_t ktiles = scale_tiles_k(FMT, a.K), qld = code_row_bytes(a.K);
    pdl_wait();
    InFlight<DT, VEC> raw[ROWS];
    load_rows<DT, VEC, ROWS>(a, unit_row<ROWS>(blockIdx.y, threadIdx.y), c, raw);
    // each factor once a block (a reciprocal costs more than the rest of a column)
    for (int i = threadIdx.y * QTX + lane; i < 16 * QTX; i += QTX * QTY) {
        const int64_t col = static_cast<int64_t>(blockIdx.x) * (16 * QTX) + i;
        float v = 1.0f;
        if (a.s != nullptr && col < a.K) v = a.weight ? __ldg(a.s + col) : recip_finite(__ldg(a.s + col));
        reinterpret_cast<float *>(&s_cs[(i & 15) >> 2][i >> 4])[i & 3] = v;
    }
    float g = 1.0f, gc = 0.0f;
    if constexpr (FMT == FMT_NV) {
        if (a.g != nullptr) g = __ldg(a.g);
        gc = __fmul_rn(recip_finite(g), 1.0f / 6.0f);
    }
    __syncthreads();
    float cs[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 t = s_cs[i][lane];
        cs[4 * i] = t.x;
        cs[4 * i + 1] = t.y;
        cs[4 * i + 2] = t.z;
        cs[4 * i + 3] = t.w;
    }
    const int64_t kt = c / TILE_K;
    const int j = (lane / LB) & 3;                          // this lane's block in its scale tile
    for (int64_t unit = blockIdx.y; unit < a.units; unit += gridDim.y) {
        const int64_t r = unit_row<ROWS>(unit, threadIdx.y);
        InFlight<DT, VEC> next[ROWS];                      // the next unit's loads run while this one is computed
        if (unit + gridDim.y < a.units) load_rows<DT, VEC, ROWS>(a, unit_row<ROWS>(unit + gridDim.y, threadIdx.y), c, next);
        if (r < a.rows) {                                   // the same for the whole warp
            uint32_t bytes = 0;                             // the rows' scales of this block
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                const int64_t row = r + 32 * u;
                if (row >= a.rows) break;
                float f[16];
                if constexpr (VEC != 0) {
                    widen16<DT>(raw[u].v, f);
                } else {
                    Raw16<DT> x;
                    settle<DT>(static_cast<const uint8_t *>(a.x) + row * a.ld * dtype_size(DT), c, a.K, raw[u].v, x);
                    widen16<DT>(x, f);
                }
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
                bytes |= block_scale<FMT>(m, gc, g, inv) << (8 * u);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 t = __fmul2_rn(make_float2(f[i], f[i + 1]), make_float2(inv, inv));
                    f[i] = t.x;
                    f[i + 1] = t.y;
                }
                if (c < 2 * qld)
                    *reinterpret_cast<uint2 *>(a.q + row * qld + (c >> 1)) = make_uint2(e2m1x8(f), e2m1x8(f + 8));
            }
            if constexpr (ROWS == 4) {
                // 4 x 4 bytes transposed over the four lanes of a scale tile:
                // lane j gets the word of row r + 32 j
                uint32_t t = __shfl_xor_sync(0xffffffffu, bytes, LB);
                bytes = __byte_perm(bytes, t, (j & 1) ? 0x3715 : 0x6240);
                t = __shfl_xor_sync(0xffffffffu, bytes, 2 * LB);
                bytes = __byte_perm(bytes, t, (j & 2) ? 0x3276 : 0x5410);
                if (lane % LB == 0 && kt < ktiles && r + 32 * j < a.rows)
                    *reinterpret_cast<uint32_t *>(a.sf + scale_word(r, kt, ktiles) + 4 * j) = bytes;
            } else {
                bytes <<= 8 * j;
                bytes |= __shfl_xor_sync(0xffffffffu, bytes, LB);
                bytes |= __shfl_xor_sync(0xffffffffu, bytes, 2 * LB);
                if (lane % (4 * LB) == 0 && kt < ktiles) *reinterpret_cast<uint32_t *>(a.sf + scale_word(r, kt, ktiles)) = bytes;
            }
        }
#pragma unroll
        for (int u = 0; u < ROWS; ++u) raw[u] = next[u];
    }
    __syncthreads();
    pdl_trigger();
}

// ---------------------------------------------------------------------------
// Values from codes: out[r, j] = RN_out(fl(e2m1(code) * scale)).  Bound by
// memory: [16384, 8192] MXFP4 -> bf16 in 56 us, 6.1 TB/s (59 without the next
// unit's loads in flight).
// ---------------------------------------------------------------------------
struct DequantArgs {
    const uint8_t *q, *sf;
    int64_t rows, K;
    const float *g;
    void *out;
    int64_t units;
};

template <int DT, int VEC, int FMT, int ROWS>
__global__ void __launch_bounds__(QTX *QTY) k_fp4_dequant(const DequantArgs a)
{
    constexpr int TILE_K = FmtT<FMT>::TILE_K, SZ = dtype_size(DT);
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * QTX + threadIdx.x) * 16;
    const int64_t ktiles = scale_tiles_k(FMT, a.K), qld = code_row_bytes(a.K);
    pdl_wait();
    const float g = (FMT == FMT_NV && a.g != nullptr) ? __ldg(a.g) : 1.0f;
    const bool in = c < a.K;
    if (VEC == 0 || in) {                                   // rows off 16 bytes take the whole warp
        const int64_t kt = c / TILE_K;
        const int shift = 8 * (static_cast<int>(c % TILE_K) / FmtT<FMT>::BLOCK);
        uint32_t words_next[ROWS] = {};                     // the rows' scale words (inside the tile, used or not)
        uint2 next[ROWS] = {};
        auto load = [&](int64_t unit) {
            const int64_t r = unit_row<ROWS>(unit, threadIdx.y);
            if (unit >= a.units || r >= a.rows || !in) return;
            if constexpr (ROWS == 4) {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(a.sf + scale_word(r, kt, ktiles)));
                words_next[0] = w.x;
                words_next[1] = w.y;
                words_next[2] = w.z;
                words_next[3] = w.w;
            } else {
                words_next[0] = __ldg(reinterpret_cast<const uint32_t *>(a.sf + scale_word(r, kt, ktiles)));
            }
#pragma unroll
            for (int u = 0; u < ROWS; ++u)
                if (r + 32 * u < a.rows) next[u] = __ldg(reinterpret_cast<const uint2 *>(a.q + (r + 32 * u) * qld + (c >> 1)));
        };
        load(blockIdx.y);
        for (int64_t unit = blockIdx.y; unit < a.units; unit += gridDim.y) {
            const int64_t r = unit_row<ROWS>(unit, threadIdx.y);
            uint32_t words[ROWS];
            uint2 q[ROWS];
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                words[u] = words_next[u];
                q[u] = next[u];
            }
            load(unit + gridDim.y);                         // runs while this unit is computed
            if (r >= a.rows) continue;
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                const int64_t row = r + 32 * u;
                if (row >= a.rows) break;
                const uint32_t b = (words[u] >> shift) & 0xffu;
                const float sc = FMT == FMT_MX ? e8m0_value(b) : __fmul_rn(e4m3_value(b), g);
                float f[16];
                e2m1x8_decode(q[u].x, f);
                e2m1x8_decode(q[u].y, f + 8);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 t = __fmul2_rn(make_float2(f[i], f[i + 1]), make_float2(sc, sc));
                    f[i] = t.x;
                    f[i + 1] = t.y;
                }
                uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.K * SZ;
                if constexpr (VEC != 0) {
                    store16<DT, VEC>(out, c, a.K, f);
                } else {
                    const int64_t c0 = c - threadIdx.x * 16;
                    store_strip<DT>(out + c0 * SZ, a.K - c0, threadIdx.x, f);
                }
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
