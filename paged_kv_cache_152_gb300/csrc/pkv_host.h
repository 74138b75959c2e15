// pkv_host.h -- host helpers that the attention entry points share: pointer
// alignment, the dynamic shared-memory limit and the caches' tensor maps.
#ifndef PKV_HOST_H
#define PKV_HOST_H

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "../../include/pkv.h"

namespace pkv {

// Raises the kernel's dynamic shared-memory limit to `smem` on the current
// device if needed.  The attribute is held per device, so what was raised is
// remembered per (device, kernel).
inline int ensure_smem_attr(const void *fn, size_t smem) {
    constexpr int kSlots = 512;
    static std::mutex mu;
    static const void *fns[kSlots];
    static int devs[kSlots];
    static size_t set[kSlots];
    static int n = 0;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    std::lock_guard<std::mutex> lock(mu);
    int k = 0;
    while (k < n && !(fns[k] == fn && devs[k] == dev)) ++k;
    if (k < n && set[k] >= smem) return PKV_OK;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    if (k == n && n < kSlots) {
        fns[n] = fn;
        devs[n] = dev;
        ++n;
    }
    if (k < kSlots) set[k] = smem;
    return PKV_OK;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// cuTensorMapEncodeTiled from the driver (looked up once, no libcuda link).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
        else
            cudaGetLastError();
    });
    return fn;
}

// The cache as a 3-D tensor: 64 dims (innermost), num_blocks * Hkv *
// block_size rows (stride head_dim * 2 bytes), head_dim / 64 halves (stride
// 128 bytes), read with the 128-byte swizzle in boxes of {64, box_rows,
// box_halves}: a box lands in shared memory as [half][row][64 dims].  No L2
// promotion: a box is one contiguous run of whole 128-byte lines already,
// and widening the requests measured ~1% slower in the decode (64 sequences
// over 50 to 900, 32 heads of 128: 96.1 against 94.8 us).
inline int encode_cache_map(CUtensorMap *map, const void *cache, int num_blocks, int num_kv_heads, int block_size,
                            int head_dim, int box_rows, int box_halves) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return PKV_ERR_CUDA;
    const cuuint64_t dims[3] = {64, (cuuint64_t)num_blocks * num_kv_heads * block_size,
                                (cuuint64_t)(head_dim / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_halves};
    const cuuint32_t elem_strides[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(cache), dims, strides,
                              box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv

#endif  // PKV_HOST_H
