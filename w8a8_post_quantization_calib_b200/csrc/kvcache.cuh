// kvcache.cuh -- the key/value cache in 8 or 4 bits: quantised as tokens are
// written into its pages, widened again as contexts are read back.
//
// A row is one token's key (or value) of one head, D elements:
//   INT8:   a = fl(max |x| / 127), code = q(fl(x * recip(a)))      value = fl(code * a)
//   FP8:    a = fl(max |x| / 448), code = e4m3(fl(x * recip(a)))   value = fl(e4m3 * a)
//   MXFP4:  blocks of 32 along D, as in fp4.cuh                    value = e2m1 * 2^(byte - 127)
// with recip as in fp4.cuh (finite).  A row that holds an infinity or a NaN
// gets the scale NaN and reads back as NaN.
//
// Cache layout: slot = page * page_size + position in the page; codes
// [slots][H][row bytes], row bytes = 16 * ceil(D / 16) (MXFP4: 16 *
// ceil(D / 32)), the padding holding zero codes, so that every row starts on
// 16 bytes; scales fp32 [slots][H], MXFP4 bytes [slots][H][ceil(D / 32)].
//
// Both kernels move bytes: a lane owns 16 elements (a 32-byte load of a
// 16-bit type), a power of two of lanes a row, so that a row's maximum is a
// few shuffles and a warp covers 32 / lanes heads of one token.
#pragma once

#include "common.cuh"
#include "fp4.cuh"
#include "ptx_sm100.cuh"

namespace sq {
namespace kv {

enum Fmt : int { KV_INT8 = 0, KV_FP8 = 1, KV_MXFP4 = 2 };

constexpr int WARPS = 8;
constexpr int MAX_D = 1024;

__host__ __device__ constexpr int row_bytes(int fmt, int D)
{
    return fmt == KV_MXFP4 ? (D + 31) / 32 * 16 : (D + 15) / 16 * 16;
}
__host__ __device__ constexpr int scale_bytes(int fmt, int D) { return fmt == KV_MXFP4 ? (D + 31) / 32 : 4; }

__device__ __forceinline__ void bad_index() { atomicCAS(&g_error_word, 0u, ERR_BAD_INDEX); }

struct WriteArgs {
    const void *k, *v;         // [T, H, D], tokens k_ld / v_ld elements apart
    int64_t T, k_ld, v_ld, num_slots;
    const int64_t *slots;      // [T]; a negative slot is skipped
    uint8_t *kc, *vc;
    void *ks, *vs;
    int H, D, groups;          // groups: warps a token (heads / heads per warp)
    int lph_log2, vec;         // lanes a row; bytes a load (32, 16, 0: single elements)
};

// NCH: chunks of 16 elements a lane (2 only for D > 512); TOK: tokens a warp,
// all their loads in flight before the first is computed.
constexpr int TOKENS = 4;

template <int DT, int FMT, int NCH, int TOK>
__global__ void __launch_bounds__(WARPS * 32) k_kv_write(const WriteArgs a)
{
    constexpr int SZ = dtype_size(DT);
    const int lane = threadIdx.x & 31, lph = 1 << a.lph_log2, sub = lane & (lph - 1);
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    const int64_t tb = unit / (2 * a.groups);
    const int rest = static_cast<int>(unit - tb * (2 * a.groups));
    const bool is_v = rest >= a.groups;
    const int h = (is_v ? rest - a.groups : rest) * (32 >> a.lph_log2) + (lane >> a.lph_log2);
    const int rb = row_bytes(FMT, a.D), sb = scale_bytes(FMT, a.D);
    pdl_wait();
    int64_t slot[TOK];
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        const int64_t t = tb * TOK + k;
        slot[k] = t < a.T ? __ldg(a.slots + t) : -1;
    }
    fp4::Raw16<DT> raw[TOK][NCH];
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        if (slot[k] >= a.num_slots) {
            if (lane == 0) bad_index();
            slot[k] = -1;
        }
        const void *src = static_cast<const uint8_t *>(is_v ? a.v : a.k) +
                          ((tb * TOK + k) * (is_v ? a.v_ld : a.k_ld) + static_cast<int64_t>(h) * a.D) * SZ;
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            fp4::load16_rt<DT>(a.vec, src, (i * lph + sub) * 16, slot[k] >= 0 && h < a.H ? a.D : 0, raw[k][i]);
    }
    uint8_t *const cache = is_v ? a.vc : a.kc;
    void *const scale = is_v ? a.vs : a.ks;
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        const bool live = slot[k] >= 0 && h < a.H;
        const int64_t row = slot[k] * a.H + h;
        float f[NCH][16];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * lph + sub) * 16;
            fp4::widen16<DT>(raw[k][i], f[i]);
            if constexpr (FMT == KV_MXFP4) m = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; j += 2) m = max3_abs_nan(m, f[i][j], f[i][j + 1]);
            if constexpr (FMT == KV_MXFP4) {
                m = max3_abs_nan(m, __shfl_xor_sync(0xffffffffu, m, 1), 0.0f);
                float inv;
                const uint32_t b = fp4::block_scale<fp4::FMT_MX>(m, 0.0f, 0.0f, inv);
#pragma unroll
                for (int j = 0; j < 16; ++j) f[i][j] = __fmul_rn(f[i][j], inv);
                if (live && c < 2 * rb) {
                    *reinterpret_cast<uint2 *>(cache + row * rb + (c >> 1)) =
                        make_uint2(fp4::e2m1x8(f[i]), fp4::e2m1x8(f[i] + 8));
                    if ((lane & 1) == 0) static_cast<uint8_t *>(scale)[row * sb + c / 32] = static_cast<uint8_t>(b);
                }
            }
        }
        if constexpr (FMT != KV_MXFP4) {
            for (int o = lph / 2; o > 0; o >>= 1) m = max3_abs_nan(m, __shfl_xor_sync(0xffffffffu, m, o), 0.0f);
            // an infinity's code times an infinite scale would be no NaN
            const float sc = m < __uint_as_float(0x7f800000u) ? scale_from_absmax_q<FMT == KV_FP8>(m)
                                                              : __uint_as_float(0x7fffffffu);
            const float inv = fp4::recip_finite(sc);
            if (live) {
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    const int c = (i * lph + sub) * 16;
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = __fmul_rn(f[i][4 * j + e], inv);
                        if constexpr (FMT == KV_FP8) w[j] = e4m3x4_bits(v[0], v[1], v[2], v[3]);
                        else w[j] = pack4_bits(quant8_bits_inrange(v[0]), quant8_bits_inrange(v[1]),
                                               quant8_bits_inrange(v[2]), quant8_bits_inrange(v[3]));
                    }
                    if (c < rb) *reinterpret_cast<uint4 *>(cache + row * rb + c) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (sub == 0) static_cast<float *>(scale)[row] = sc;
            }
        }
    }
    __syncthreads();
    pdl_trigger();
}

struct ReadArgs {
    const uint8_t *kc, *vc;
    const void *ks, *vs;
    int64_t num_pages, max_pages;      // max_pages: columns of the table
    const int32_t *table;              // [B, max_pages]
    const int32_t *cu;                 // [B + 1]: first output row of each sequence
    const int32_t *starts;             // [B] or null (0): position of each sequence's first row
    int64_t total;                     // rows of the outputs
    void *k, *v;                       // [total, H, D]
    int B, H, D, groups, page_size;
    int lph_log2, vec;
};

// Largest b in [0, B) with cu[b] <= t (-1 when t lies behind cu[B] or before
// cu[0]): the warp's lanes probe 32 points at a time.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int B, int64_t t, int lane)
{
    int lo = 0, n = B + 1;             // cu[lo] .. cu[lo + n - 1] remain
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, at < n && __ldg(cu + lo + at) <= t);
        if (le == 0) return -1;
        const int last = 31 - __clz(le);
        if (step == 1) {
            lo += last;
            break;
        }
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo < B ? lo : -1;
}

template <int DT, int FMT, int NCH, int TOK>
__global__ void __launch_bounds__(WARPS * 32) k_kv_read(const ReadArgs a)
{
    constexpr int SZ = dtype_size(DT);
    const int lane = threadIdx.x & 31, lph = 1 << a.lph_log2, sub = lane & (lph - 1);
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    const int64_t t0 = unit / a.groups * TOK;
    const int h = static_cast<int>(unit % a.groups) * (32 >> a.lph_log2) + (lane >> a.lph_log2);
    const int rb = row_bytes(FMT, a.D), sb = scale_bytes(FMT, a.D);
    pdl_wait();
    // the sequence of the first token; the others follow it or start a later one
    int64_t row[TOK];                  // row of the cache, -1: zeros, -2: the output row is left as it was
    int b = -1;
    int64_t first = 0, end = 0, start = 0;                 // of sequence b
    const int64_t total = min(a.total, static_cast<int64_t>(__ldg(a.cu + a.B)));
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        const int64_t t = t0 + k;
        row[k] = -2;
        if (t >= total) continue;                          // the same for the whole warp
        if (b < 0 || t >= end) {
            b = sequence_of(a.cu, a.B, t, lane);
            if (b < 0) continue;
            first = __ldg(a.cu + b);
            end = __ldg(a.cu + b + 1);
            start = a.starts != nullptr ? __ldg(a.starts + b) : 0;
        }
        const int64_t pos = t - first + start;
        const int64_t pi = pos / a.page_size;
        const int64_t page = pos >= 0 && pi < a.max_pages ? __ldg(a.table + b * a.max_pages + pi) : -1;
        if (page >= 0 && page < a.num_pages) {
            row[k] = (page * a.page_size + (pos - pi * a.page_size)) * a.H + h;
        } else {
            row[k] = -1;
            if (lane == 0) bad_index();
        }
    }
    if (h < a.H) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * lph + sub) * 16;
            if (c >= a.D) break;
            uint4 q[TOK][2];
            float sc[TOK][2];
#pragma unroll
            for (int k = 0; k < TOK; ++k) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const uint8_t *cache = n ? a.vc : a.kc;
                    const void *scale = n ? a.vs : a.ks;
                    q[k][n] = make_uint4(0u, 0u, 0u, 0u);
                    sc[k][n] = 0.0f;
                    if (row[k] >= 0) {
                        if constexpr (FMT == KV_MXFP4) {
                            const uint2 t2 = __ldg(reinterpret_cast<const uint2 *>(cache + row[k] * rb + (c >> 1)));
                            q[k][n].x = t2.x;
                            q[k][n].y = t2.y;
                            sc[k][n] = fp4::e8m0_value(__ldg(static_cast<const uint8_t *>(scale) + row[k] * sb + c / 32));
                        } else {
                            q[k][n] = __ldg(reinterpret_cast<const uint4 *>(cache + row[k] * rb + c));
                            sc[k][n] = __ldg(static_cast<const float *>(scale) + row[k]);
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < TOK; ++k) {
                if (row[k] == -2) continue;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float f[16];
                    if constexpr (FMT == KV_MXFP4) {
                        fp4::e2m1x8_decode(q[k][n].x, f);
                        fp4::e2m1x8_decode(q[k][n].y, f + 8);
                    } else {
                        const uint32_t w[4] = {q[k][n].x, q[k][n].y, q[k][n].z, q[k][n].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (FMT == KV_INT8) {
                                // 2^23 + (code + 128) has the code's byte in its low bits
                                const uint32_t u = w[j] ^ 0x80808080u;
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    f[4 * j + e] = __fsub_rn(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + e)), 8388736.0f);
                            } else {
                                uint32_t h2[2];
                                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2[0]) : "h"(static_cast<uint16_t>(w[j])));
                                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2[1]) : "h"(static_cast<uint16_t>(w[j] >> 16)));
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&h2[e]));
                                    f[4 * j + 2 * e] = p.x;
                                    f[4 * j + 2 * e + 1] = p.y;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) f[j] = __fmul_rn(f[j], sc[k][n]);
                    fp4::store16_rt<DT>(a.vec, static_cast<uint8_t *>(n ? a.v : a.k) + ((t0 + k) * a.H + h) * a.D * SZ, c, a.D, f);
                }
            }
        }
    }
    __syncthreads();
    pdl_trigger();
}

}  // namespace kv
}  // namespace sq
