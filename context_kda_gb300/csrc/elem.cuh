// Element types of the operators around the KDA layer: activations in bf16, fp16 or fp32, computed in
// fp32.  Rounding to the activation type happens once, at the store (round to nearest even).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename E> __device__ __forceinline__ E from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Bytes of an element type code (0: not a type).
inline int elem_bytes(int32_t type)
{
    return type == KDA_TYPE_F32 ? 4 : (type == KDA_TYPE_BF16 || type == KDA_TYPE_F16) ? 2 : 0;
}

}  // namespace kda
