// Elements of the 16- and 32-bit float types.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_ptx.cuh"

namespace gct {
namespace fp8 {

enum : int { T_F16 = 0, T_BF16 = 1, T_F32 = 2 };

template <int T>
__device__ __forceinline__ float load_elem(const void* p, long long i) {
    if (T == T_F32) return static_cast<const float*>(p)[i];
    if (T == T_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <int T>
__device__ __forceinline__ void unpack16(uint32_t w, float& lo, float& hi) {
    if (T == T_F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        lo = f.x;
        hi = f.y;
    } else {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t pack16(float a, float b, int bf16) {
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace fp8
}  // namespace gct
