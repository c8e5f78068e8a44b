// Tensor maps (host) and the tiled TMA loads that use them (device), plus a
// bounded mbarrier wait; shared by the paged and the prompt attention.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "tma_ptx.cuh"

namespace kvo {

// cuTensorMapEncodeTiled is looked up through the runtime (the library does not link libcuda).
//
// Host: `dims` dimensions, innermost first; strides[i] is the byte stride of dimension i + 1.  The box's
// inner extent in bytes picks the swizzle (128 or 64).  Out-of-range elements read as zero.
inline bool tensor_map(CUtensorMap* m, const void* base, int elem, int dims, const uint64_t* sizes,
                       const uint64_t* strides, const uint32_t* box) {
    typedef CUresult (*Enc)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<void*> encoder{nullptr};
    void* f = encoder.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess || !f) {
            cudaGetLastError();
            return false;
        }
        encoder.store(f, std::memory_order_release);
    }
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    const uint32_t inner = box[0] * elem;
    return ((Enc)f)(m, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims,
                    const_cast<void*>(base), (const cuuint64_t*)sizes, (const cuuint64_t*)strides,
                    (const cuuint32_t*)box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Host: `rows` contiguous rows of d elements; boxes of box_bytes x box_rows.
inline bool tensor_map_rows(CUtensorMap* m, const void* base, int elem, int d, uint64_t rows, int box_bytes,
                            int box_rows) {
    const uint64_t sizes[2] = {(uint64_t)d, rows};
    const uint64_t strides[1] = {(uint64_t)d * elem};
    const uint32_t box[2] = {(uint32_t)(box_bytes / elem), (uint32_t)box_rows};
    return tensor_map(m, base, elem, 2, sizes, strides, box);
}

__device__ __forceinline__ void tensor_map_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(mbar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar)
        : "memory");
}

// Waits for the phase of the given parity to complete, for at most limit_ns; false when the limit passed.
__device__ __forceinline__ bool mbar_wait_bounded(uint32_t mbar, uint32_t parity, long long limit_ns) {
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(mbar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(mbar, parity))
        if ((long long)(global_ns() - t0) > limit_ns) return false;
    return true;
}

}  // namespace kvo
