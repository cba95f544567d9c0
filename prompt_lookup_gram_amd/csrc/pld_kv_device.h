// Device helpers that the cache's writers share: rotations, words of 8
// elements, and V stored along its positions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pld_target_device.h"

namespace pld {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;   // head_dim 256
constexpr int kSpan = 64;        // positions of a V tile
constexpr int kPad = 2;          // elements between rows of the V tile

typedef uint32_t U4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void turn(double turns, int32_t p, float gain, float &c, float &s)
{
    const double x = turns * p;
    sincospif((float)(2.0 * (x - rint(x))), &s, &c);
    c *= gain;
    s *= gain;
}

// 8 elements of T.
template <typename T>
struct Eight {
    T x[8];
};

template <typename T>
__device__ __forceinline__ Eight<T> load8(const T *p)
{
    return __builtin_bit_cast(Eight<T>, *(const U4 *)p);
}

// Stores 8 values rounded to C: 16 or 8 bytes.
template <typename C>
__device__ __forceinline__ void store8(C *p, const float (&y)[8])
{
    Eight<C> w;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w.x[i] = from_f32<C>(y[i]);
    struct __attribute__((aligned(8 * sizeof(C)))) Out {
        Eight<C> w;
    };
    *(Out *)p = Out{w};
}

// Stores V of one tile of kSpan positions of one request and kv head; `id`
// counts kv heads first, then tiles, then requests.
template <typename T, typename C>
__device__ __forceinline__ void store_values(const KvAppendArgs &a, uint32_t id, uint32_t tiles,
                                             char *lds)
{
    const BlockArgs &g = a.blk;
    const int32_t dim = g.head_dim, tokens = 1 << g.page_shift, tid = threadIdx.x;
    int32_t length;
    uint32_t err;
    const int32_t h = id % (uint32_t)g.kv_heads;
    const uint32_t bt = id / (uint32_t)g.kv_heads;
    const int32_t b = bt / tiles;
    const int32_t n = block_rows(g, b, length, err);
    if (n <= 0)
        return;
    // the tile's positions, and those of them the block has
    const int64_t p0 = ((int64_t)(length - 1) / kSpan + bt % tiles) * kSpan;
    const int64_t from = p0 > length - 1 ? p0 : length - 1;
    const int64_t last = (int64_t)length - 1 + n;
    const int64_t to = p0 + kSpan < last ? p0 + kSpan : last;
    if (from >= to)
        return;
    T *tile = (T *)lds;
    const int32_t pitch = dim + kPad, words = dim / 8;
    const T *v = (const T *)a.v + ((int64_t)b * g.rows - (length - 1)) * a.kv_stride +
                 (int64_t)h * dim;
    // (a thread stores the same 8 positions of every dim it takes)
    static_assert(kThreads % (kSpan / 8) == 0, "");
    const int32_t at = tid % (kSpan / 8) * 8;
    const int64_t first = p0 + at;
    const bool any = first + 8 > from && first < to;
    const bool whole = first >= from && first + 8 <= to;
    const int32_t page = any ? page_of(g, b, (int32_t)(first > from ? first : from)) : -1;
    for (int32_t i = tid; i < (int32_t)(to - from) * words; i += kThreads) {
        const int64_t p = from + i / words;
        const int32_t d = i % words * 8;
        const Eight<T> x = load8(v + p * a.kv_stride + d);
        T *row = tile + (int32_t)(p - p0) * pitch + d;
        // (rows are padded: 4 bytes at a time)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            ((uint32_t *)row)[k] = __builtin_bit_cast(U4, x)[k];
    }
    __syncthreads();
    const float scale = g.v_scale ? g.v_scale[h] : 1.0f;
    if (page < 0)
        return;  // (a bad page is reported by the row's K)
    for (int32_t i = tid; i < kSpan / 8 * dim; i += kThreads) {
        const int32_t d = i / (kSpan / 8);
        C *out = (C *)a.v_cache + (((int64_t)page * g.kv_heads + h) * dim + d) * tokens +
                 (first & (tokens - 1));
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            y[k] = whole || (first + k >= from && first + k < to)
                       ? to_f32(tile[(at + k) * pitch + d]) / scale
                       : 0.0f;
        if (whole) {
            store8<C>(out, y);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (first + k >= from && first + k < to)
                    out[k] = from_f32<C>(y[k]);
        }
    }
}

}  // namespace

}  // namespace pld
