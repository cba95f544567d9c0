// Device helpers shared by the verify step's kernels: element types, the
// rows of a request's block and page lookups.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pld.h"
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

// The rows of request b's block: 0 when it has none, -1 when its inputs are
// bad (the sticky bits are returned in `err`).
__device__ __forceinline__ int32_t block_rows(const BlockArgs &a, int32_t b, int32_t &length,
                                              uint32_t &err)
{
    length = a.lengths[b];
    const int32_t d = a.draft_len[b];
    err = 0;
    if (length < 0)
        err |= kErrLenNegative;
    if (d < -1 || d >= a.rows)
        err |= kErrBlock;
    if (err)
        return -1;
    if (length == 0 || d == -1)
        return 0;
    if ((int64_t)length + d > a.max_len) {
        err |= kErrLenCapacity;
        return -1;
    }
    return d + 1;
}

// The page that holds position `pos` of request b, or -1 when it is bad.
__device__ __forceinline__ int32_t page_of(const BlockArgs &a, int32_t b, int32_t pos)
{
    const int64_t i = pos >> a.page_shift;
    if (i >= a.table_stride)
        return -1;
    const int32_t id = a.table[(int64_t)b * a.table_stride + i];
    return (uint32_t)id < (uint64_t)a.n_pages ? id : -1;
}

}  // namespace pld
