// tma_slabs.cuh -- one TMA load for a whole tile of rows wider than a 128-byte swizzle: the row's
// slabs of 64 elements are a dimension of the tensor map.
#pragma once

#include "tc_ptx.cuh"
#include "tmap.h"

namespace efla {
namespace tc {

__device__ __forceinline__ void tma_load_4d(void *dst, const void *map, uint64_t *bar, int c0,
                                            int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

}  // namespace tc

namespace tmap {

// 16-bit tensor [d2][d1][64 slabs] as (64, d1, slabs, d2) with a (64, b1, slabs, 1) box: one load brings every
// 64-element slab of b1 rows, slab after slab.
inline bool make_slabs(CUtensorMap *m, const void *ptr, uint32_t slabs, uint64_t d1, uint64_t d2, uint32_t b1,
                       CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t row = (cuuint64_t)slabs * 128;
    const cuuint64_t dims[4] = {64, d1, slabs, d2};
    const cuuint64_t strides[3] = {row, 128, row * d1};
    const cuuint32_t box[4] = {64, b1, slabs, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, dt, 4, const_cast<void *>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tmap
}  // namespace efla
