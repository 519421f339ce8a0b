// element.cuh -- single elements of 16- and 32-bit floats, by type code.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace dtc {

// ------------------------------------------------------------------------------------------------
// Elements of a 16- or 32-bit float type by code: 0 bf16, 1 fp16, 2 fp32
// ------------------------------------------------------------------------------------------------
template <int kType>
__device__ __forceinline__ float load_f(const void* p, int64_t i) {
    if constexpr (kType == 0) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    else if constexpr (kType == 1) return __half2float(static_cast<const __half*>(p)[i]);
    else return static_cast<const float*>(p)[i];
}
template <int kType>
__device__ __forceinline__ void store_f(void* p, int64_t i, float v) {
    if constexpr (kType == 0) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else if constexpr (kType == 1) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<float*>(p)[i] = v;
}
__device__ __forceinline__ float load_w(const void* p, int64_t i, int type) {
    return type == 0 ? load_f<0>(p, i) : type == 1 ? load_f<1>(p, i) : load_f<2>(p, i);
}
__device__ __forceinline__ void store_w(void* p, int64_t i, float v, int type) {
    if (type == 0) store_f<0>(p, i, v);
    else if (type == 1) store_f<1>(p, i, v);
    else store_f<2>(p, i, v);
}

}  // namespace dtc
