// Device helpers shared by the verify step's kernels: element types (and, from
// pld_block.h, the rows of a request's block and page lookups).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pld.h"
#include "pld_block.h"
#include "pld_kernels.h"
#include "pld_target.h"

namespace pld {

// 8-bit cache cells (PLD_E4M3), as raw bytes.
struct E4m3 {
    uint8_t bits;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(__bf16 x)
{
    return __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(uint16_t, x) << 16);
}
__device__ __forceinline__ float to_f32(E4m3 x)
{
    return __builtin_amdgcn_cvt_f32_fp8((int)x.bits, 0);
}

// Round to the nearest value of T, ties to even; an 8-bit cell saturates at
// 448 (the conversion instruction would give NaN) and keeps NaN.
template <typename T>
__device__ __forceinline__ T from_f32(float x)
{
    return (T)x;
}
template <>
__device__ __forceinline__ E4m3 from_f32<E4m3>(float x)
{
    const float c = x > 448.0f ? 448.0f : (x < -448.0f ? -448.0f : x);
    return E4m3{(uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(c, c, 0, false) & 0xff)};
}

}  // namespace pld
