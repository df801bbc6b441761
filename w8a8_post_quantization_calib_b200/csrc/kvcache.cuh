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
// The three kernels move bytes: a lane owns 16 elements (a 32-byte access of a
// 16-bit type).
//   k_kv_write      rows of all tokens end to end, a power of two of lanes a
//                   row, so that a row's maximum is a few shuffles (heads of 80
//                   or 96 leave lanes idle)
//   k_kv_read       a warp, or several, a token; the same lanes a row
//   k_kv_read_rows  rows end to end, ceil(D / 16) lanes a row
// 8 heads of 128 bf16: 10.3 k tokens written as E4M3 in 13.3 us (64 MB, 4.8
// TB/s) and read back in 13.1; contexts of 75 k tokens read back from MXFP4 in
// 69.2 us (400 MB, 5.8 TB/s of 6.57 copied), from INT8 in 87.  A decode step's
// 64 tokens take 1.7 and 2.7 us: launches and chains of loads.
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

// 1 once a kernel met an index of the caller outside the cache (the access was
// skipped).  Apart from g_error_word, so that it hides no barrier timeout.
static __device__ unsigned int g_bad_index;

__device__ __forceinline__ void bad_index() { atomicExch(&g_bad_index, 1u); }

struct WriteArgs {
    const void *k, *v;         // [T, H, D], tokens k_ld / v_ld elements apart
    int64_t T, k_ld, v_ld, num_slots;
    const int64_t *slots;      // [T]; a negative slot is skipped
    uint8_t *kc, *vc;
    void *ks, *vs;
    int H, D;
    int lph_log2, vec;         // lanes a row; bytes a load (32, 16, 8, 4, 0: single elements)
    uint64_t head_inv;         // ceil(2^63 / H): division by a product
};

// Rows (token, head) laid end to end, 32 / lanes of them a step; keys and values
// in turn by warps.  NCH: chunks of 16 elements a lane (2 only for D > 512); TOK:
// steps a warp, all their loads in flight before the first is computed.
constexpr int TOKENS = 2;

template <int DT, int FMT, int VEC, int NCH, int TOK>
__global__ void __launch_bounds__(WARPS * 32) k_kv_write(const WriteArgs a)
{
    constexpr int SZ = dtype_size(DT);
    const int lane = threadIdx.x & 31, lph = 1 << a.lph_log2, sub = lane & (lph - 1), per = 32 >> a.lph_log2;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    const bool is_v = unit & 1;
    const int64_t rows = a.T * a.H;
    const int rb = row_bytes(FMT, a.D), sb = scale_bytes(FMT, a.D);
    pdl_wait();
    // the loads do not wait for the slots: a skipped token's row is read all the same
    fp4::Raw16<DT> raw[TOK][NCH];
    int64_t slot[TOK];
    int h[TOK];
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        const int64_t r = ((unit >> 1) * TOK + k) * per + (lane >> a.lph_log2);
        // r < 2^47 and H <= 2^16: the error of the quotient, r / 2^63, is below 1 / H
        const int64_t t = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(r) << 1, a.head_inv));
        h[k] = static_cast<int>(r - t * a.H);
        slot[k] = r < rows ? __ldg(a.slots + t) : -1;
        const void *src = static_cast<const uint8_t *>(is_v ? a.v : a.k) +
                          (t * (is_v ? a.v_ld : a.k_ld) + static_cast<int64_t>(h[k]) * a.D) * SZ;
#pragma unroll
        for (int i = 0; i < NCH; ++i) fp4::load16_rt<DT, VEC>(a.vec, src, (i * lph + sub) * 16, r < rows ? a.D : 0, raw[k][i]);
    }
    uint8_t *const cache = is_v ? a.vc : a.kc;
    void *const scale = is_v ? a.vs : a.ks;
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        if (slot[k] >= a.num_slots && sub == 0) bad_index();
        const bool live = slot[k] >= 0 && slot[k] < a.num_slots;
        const int64_t row = slot[k] * a.H + h[k];
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
    int part_log2;                     // warps a token (a power of two)
    uint64_t page_inv, head_inv;       // ceil(2^63 / page_size), ceil(2^63 / H): division by a product
    int lanes;                         // k_kv_read_rows: lanes a row
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

// The page that holds position `pos` of sequence b (-1: outside the table), and
// its column pi.  Output rows and starts are below 2^31, so positions are below
// 2^32 (with a first row below 0 they can be higher: outside); page_size < 2^31,
// so the quotient's error, pos / 2^63, is below 1 / page_size.
__device__ __forceinline__ int64_t page_of(const ReadArgs &a, int b, int64_t pos, int64_t &pi)
{
    pi = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(pos) << 1, a.page_inv));
    return (static_cast<uint64_t>(pos) >> 32) == 0 && pi < a.max_pages ? __ldg(a.table + b * a.max_pages + pi) : -1;
}

// 16 codes of a row and their scale
template <int FMT>
__device__ __forceinline__ void load_codes(const uint8_t *cache, const void *scale, int64_t row, int rb, int sb, int c,
                                           uint4 &q, uint32_t &sc)
{
    if constexpr (FMT == KV_MXFP4) {
        const uint2 t = __ldg(reinterpret_cast<const uint2 *>(cache + row * rb + (c >> 1)));
        q.x = t.x;
        q.y = t.y;
        sc = __ldg(static_cast<const uint8_t *>(scale) + row * sb + c / 32);
    } else {
        q = __ldg(reinterpret_cast<const uint4 *>(cache + row * rb + c));
        sc = __ldg(static_cast<const uint32_t *>(scale) + row);
    }
}

template <int FMT>
__device__ __forceinline__ void widen_codes(const uint4 &q, uint32_t scale, float (&f)[16])
{
    const float sc = FMT == KV_MXFP4 ? fp4::e8m0_value(scale) : __uint_as_float(scale);
    if constexpr (FMT == KV_MXFP4) {
        fp4::e2m1x8_decode(q.x, f);
        fp4::e2m1x8_decode(q.y, f + 8);
    } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
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
    for (int j = 0; j < 16; ++j) f[j] = __fmul_rn(f[j], sc);
}

// A warp (of 2^part_log2) reads one output row: it finds where the row lies, a
// chain of dependent loads, and streams its heads with U groups of keys and
// values in flight.
template <int DT, int FMT, int VEC>
__global__ void __launch_bounds__(WARPS * 32) k_kv_read(const ReadArgs a)
{
    constexpr int SZ = dtype_size(DT), U = 2;
    const int lane = threadIdx.x & 31, lph = 1 << a.lph_log2, sub = lane & (lph - 1);
    const int rb = row_bytes(FMT, a.D), sb = scale_bytes(FMT, a.D);
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    const int64_t t = unit >> a.part_log2;
    const int part = static_cast<int>(unit & ((1 << a.part_log2) - 1));
    pdl_wait();
    const int b = t < a.total ? sequence_of(a.cu, a.B, t, lane) : -1;
    if (b >= 0) {
        const int64_t pos = t - __ldg(a.cu + b) + (a.starts != nullptr ? __ldg(a.starts + b) : 0);
        int64_t pi;
        const int64_t page = page_of(a, b, pos, pi);
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok && lane == 0) bad_index();
        const int64_t row0 = (page * a.page_size + (pos - pi * a.page_size)) * a.H, out0 = t * a.H;
        for (int g = part; g < a.groups; g += U << a.part_log2) {
            for (int c = sub * 16; c < a.D; c += lph * 16) {             // more than once for D > 512 only
                uint4 q[U][2] = {};
                uint32_t sc[U][2] = {};
                int h[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    h[u] = (g + (u << a.part_log2)) * (32 >> a.lph_log2) + (lane >> a.lph_log2);
                    if (ok && h[u] < a.H) {
                        load_codes<FMT>(a.kc, a.ks, row0 + h[u], rb, sb, c, q[u][0], sc[u][0]);
                        load_codes<FMT>(a.vc, a.vs, row0 + h[u], rb, sb, c, q[u][1], sc[u][1]);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (h[u] >= a.H) continue;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        float f[16];
                        widen_codes<FMT>(q[u][n], sc[u][n], f);
                        fp4::store16_rt<DT, VEC>(a.vec, static_cast<uint8_t *>(n ? a.v : a.k) + (out0 + h[u]) * a.D * SZ, c, a.D, f);
                    }
                }
            }
        }
    }
    __syncthreads();
    pdl_trigger();
}

// Rows whose lanes are no power of two, or fewer heads than a warp has rows:
// output rows (token, head) laid end to end, 32 / lanes of them a step, U steps
// a warp.  Every lane finds its own row's place, starting from the sequence of
// the warp's first token.  D <= 512.
template <int DT, int FMT, int VEC>
__global__ void __launch_bounds__(WARPS * 32) k_kv_read_rows(const ReadArgs a)
{
    constexpr int SZ = dtype_size(DT), U = 2;
    const int lane = threadIdx.x & 31;
    const int per = 32 / a.lanes, j = lane / a.lanes, c = (lane - j * a.lanes) * 16;
    const int rb = row_bytes(FMT, a.D), sb = scale_bytes(FMT, a.D);
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    const int64_t r0 = unit * (U * per), rows = a.total * a.H;
    // r < 2^47 and H <= 2^16: the error of the quotient, r / 2^63, is below 1 / H
    auto token = [&](int64_t r) { return static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(r) << 1, a.head_inv)); };
    pdl_wait();
    if (r0 < rows) {
        const int b0 = max(sequence_of(a.cu, a.B, token(r0), lane), 0);
        const int64_t first0 = __ldg(a.cu + b0), end0 = __ldg(a.cu + b0 + 1);
        const int64_t start0 = a.starts != nullptr ? __ldg(a.starts + b0) : 0;
        int64_t row[U];                // row of the cache, -1: outside (zeros), -2: the output row stays
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * per + j, t = token(r);
            row[u] = -2;
            if (j >= per || r >= rows) continue;
            int b = b0;
            int64_t first = first0, end = end0, start = start0;
            if (t >= end && b + 1 < a.B) {
                int step = 1;                               // the answer lies before b + step
                while (b + step < a.B && __ldg(a.cu + b + step) <= t) {
                    b += step;
                    step = min(2 * step, a.B);
                }
                while (step > 1) {
                    step = (step + 1) / 2;
                    if (b + step < a.B && __ldg(a.cu + b + step) <= t) b += step;
                }
                first = __ldg(a.cu + b);
                end = __ldg(a.cu + b + 1);
                start = a.starts != nullptr ? __ldg(a.starts + b) : 0;
            }
            if (t < first || t >= end) continue;
            const int64_t pos = t - first + start;
            int64_t pi;
            const int64_t page = page_of(a, b, pos, pi);
            if (page >= 0 && page < a.num_pages) {
                row[u] = (page * a.page_size + (pos - pi * a.page_size)) * a.H + (r - t * a.H);
            } else {
                row[u] = -1;
                bad_index();
            }
        }
        uint4 q[U][2] = {};
        uint32_t sc[U][2] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row[u] >= 0) {
                load_codes<FMT>(a.kc, a.ks, row[u], rb, sb, c, q[u][0], sc[u][0]);
                load_codes<FMT>(a.vc, a.vs, row[u], rb, sb, c, q[u][1], sc[u][1]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row[u] == -2) continue;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float f[16];
                widen_codes<FMT>(q[u][n], sc[u][n], f);
                fp4::store16_rt<DT, VEC>(a.vec, static_cast<uint8_t *>(n ? a.v : a.k) + (r0 + u * per + j) * a.D * SZ, c, a.D, f);
            }
        }
    }
    __syncthreads();
    pdl_trigger();
}

}  // namespace kv
}  // namespace sq
