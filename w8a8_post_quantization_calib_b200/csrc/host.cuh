// host.cuh -- host-side helpers shared by the translation units of libsq:
// argument checks, per-device figures, launches (programmatic dependent
// launch, clusters), dynamic shared memory and TMA tensor maps.
#pragma once

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>
#include <unordered_map>
#include <utility>

#include "sq.h"
#include "common.cuh"

namespace sq {

inline thread_local int t_last_cuda_error = 0;
inline unsigned long long g_timeout_ns = 2000000000ull;   // bounded barrier waits: 2 s
inline int g_inject = 0;                                // failure-detection test knob

constexpr int kMaxDevices = 64;
inline int g_sm_count[kMaxDevices] = {0};
inline std::mutex g_mu;

inline cudaStream_t as_stream(sq_stream s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool valid_dt(int dt) { return dt == SQ_F32 || dt == SQ_F16 || dt == SQ_BF16; }

inline sq_status cuda_fail(cudaError_t e)
{
    t_last_cuda_error = static_cast<int>(e);
    return SQ_ERR_CUDA;
}

inline sq_status check_launch()
{
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SQ_OK : cuda_fail(e);
}

inline int sm_count()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    if (g_sm_count[dev] == 0) {
        int n = 0;
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        g_sm_count[dev] = n > 0 ? n : 148;
    }
    return g_sm_count[dev];
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Programmatic dependent launch is used only on explicitly created streams;
// on the legacy and per-thread default streams launches go without the
// attribute (plain stream order), which is where the chains that first showed
// the early-trigger hazard (see pdl_wait in common.cuh) ran.
inline bool pdl_stream(cudaStream_t st)
{
    return st != nullptr && st != cudaStreamLegacy && st != cudaStreamPerThread;
}

// Launch with programmatic stream serialisation (see pdl_wait in common.cuh):
// the kernel may begin while the previous kernel of the stream drains.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_stream(st) ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// launch_pdl with a runtime cluster shape (cluster_x CTAs along x) and
// dynamic shared memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster_smem(void (*kern)(KArgs...), dim3 grid, dim3 block, unsigned cluster_x, size_t smem,
                                    cudaStream_t st, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster_x;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_stream(st) ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// launch_pdl with a runtime cluster shape (cluster_x CTAs along x).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, unsigned cluster_x, cudaStream_t st,
                               Args &&...args)
{
    return launch_pdl_cluster_smem(kern, grid, block, cluster_x, 0, st, std::forward<Args>(args)...);
}

// Per (device, kernel): dynamic shared memory already granted, and the
// occupancy figures the launch sizes its grid with.  Queried once.
struct KernelInfo {
    int smem_set = 0;
    int per_sm = 0;           // resident blocks per SM with per_sm_smem bytes of dynamic shared memory
    int per_sm_smem = -1;
    int clusters = 0;
};
inline std::unordered_map<uint64_t, KernelInfo> g_kinfo;

inline KernelInfo &kinfo(const void *kern)
{
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t key = (static_cast<uint64_t>(dev) << 56) ^ reinterpret_cast<uint64_t>(kern);
    return g_kinfo[key];
}

// Grants `smem` bytes of dynamic shared memory to `kern` (once per size increase).
inline cudaError_t ensure_smem(const void *kern, int smem)
{
    std::lock_guard<std::mutex> lk(g_mu);
    KernelInfo &ki = kinfo(kern);
    if (ki.smem_set >= smem) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) ki.smem_set = smem;
    return e;
}

// ------------------------------------------------------------------ TMA maps
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::lock_guard<std::mutex> lk(g_mu);
    if (fn == nullptr) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}

// 2D row-major [rows, inner] tensor of 1- or 2-byte elements; box of
// box_rows x 128 bytes with the 128-byte swizzle; out-of-range reads are zero.
inline bool make_map(CUtensorMap *m, const void *base, bool f16, int64_t inner, int64_t rows, uint32_t box_rows)
{
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const int elt = f16 ? 2 : 1;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(inner * elt)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elt), box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                          const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 3D view of a row-major [rows, K] int8 tensor (K a multiple of 128) as
// [K/128][rows][128 bytes]: box = box_rows x 128 bytes x kbo blocks, each
// block landing as its own 128-byte-swizzled tile.
inline bool make_map3(CUtensorMap *m, const void *base, int64_t K, int64_t rows, uint32_t box_rows, uint32_t kbo)
{
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(K / 128)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(K), 128};
    cuuint32_t box[3] = {128, box_rows, kbo};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Output map for the epilogue's TMA stores: [M, N] row-major, 32 x 32 boxes,
// swizzle matching the staging layout (64-byte rows for 2-byte elements,
// 128-byte rows for 4-byte ones).
inline bool make_out_map(CUtensorMap *m, void *base, int out_dt, bool s32, int64_t M, int64_t N)
{
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    CUtensorMapDataType t;
    int elt;
    if (s32) { t = CU_TENSOR_MAP_DATA_TYPE_INT32; elt = 4; }
    else if (out_dt == SQ_F32) { t = CU_TENSOR_MAP_DATA_TYPE_FLOAT32; elt = 4; }
    else if (out_dt == SQ_F16) { t = CU_TENSOR_MAP_DATA_TYPE_FLOAT16; elt = 2; }
    else { t = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16; elt = 2; }
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(N * elt)};
    cuuint32_t box[2] = {32, 32};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, t, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          elt == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Each translation unit has its own device error word (common.cuh); this
// reads and clears the current device's words of libsq_fp4.cu: the barrier
// timeout and the key/value cache's bad index.
cudaError_t fp4_error_words_take(unsigned int *timeout, unsigned int *bad_index);
inline std::atomic<bool> g_fp4_launched{false};   // a call that can set one of them was made

}  // namespace sq
