// The rows of a request's block and page lookups of the verify step: every
// index that the kernels form from lengths, draft lengths and page tables is
// checked here. Plain C++, so that a host test can run it under sanitizers.
#pragma once

#include <stdint.h>

#include "pld_kernels.h"
#include "pld_target.h"

#ifdef __HIPCC__
#define PLD_INLINE __device__ __forceinline__
#else
#define PLD_INLINE inline
#endif

namespace pld {

// The rows of request b's block: 0 when it has none, -1 when its inputs are
// bad (the sticky bits are returned in `err`).
PLD_INLINE int32_t block_rows(const BlockArgs &a, int32_t b, int32_t &length,
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
PLD_INLINE int32_t page_of(const BlockArgs &a, int32_t b, int32_t pos)
{
    const int64_t i = pos >> a.page_shift;
    if (i >= a.table_stride)
        return -1;
    const int32_t id = a.table[(int64_t)b * a.table_stride + i];
    return (uint32_t)id < (uint64_t)a.n_pages ? id : -1;
}

}  // namespace pld
