// Two 16-bit numbers to a 32-bit word, and back.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "w4a16.h"

namespace w4a16 {

template <int DTYPE>
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b)
{
    if constexpr (DTYPE == W4A16_BF16) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        a = f.x;
        b = f.y;
    }
}

template <int DTYPE>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (DTYPE == W4A16_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

}  // namespace w4a16
