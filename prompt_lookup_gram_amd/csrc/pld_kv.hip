// Rotary positions and the paged cache's writer, for gfx950 (MI355X).
//
// Mathematics: a pair (x, y) at position p becomes g (x cos a - y sin a,
// x sin a + y cos a), a = p f. The angle is kept in turns, as a 64-bit product
// whose whole part is dropped (at position 262,144 a 32-bit product would be
// off by 2^-6 radians); sine and cosine of the rest are 32-bit.
//
// Bound by memory: every element is read and written once. A row's angles
// are the same for all its heads, so a workgroup computes them once into LDS
// and then streams the heads in 16-byte words. V pages hold positions side by
// side: a workgroup collects 64 positions of a head in LDS and stores them
// along the positions, 16 bytes at a time where 8 positions are its own.
// 65,536 rows of 32 + 8 + 8 heads of 128 in bf16: 325 us, 4.9 TB/s read and
// written (a large copy reaches 4.8); 1,149 us an element at a time.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pld_kv_device.h"

namespace pld {

namespace {

constexpr int64_t kManyRows = 1536;  // from which on a workgroup takes 4 of them

// Words of 8 elements: q, k and v 16-byte aligned with strides of 8 elements,
// and rotated pairs that fill whole words.
//
// The first `turning` workgroups rotate R rows each, the others store V: one
// per request, kv head and tile of kSpan positions.
template <typename T, typename C, int R>
__global__ __launch_bounds__(kThreads) void append_words(KvAppendArgs a, uint32_t turning,
                                                         uint32_t tiles)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const BlockArgs &g = a.blk;
    const int32_t dim = g.head_dim, tokens = 1 << g.page_shift, tid = threadIdx.x;
    int32_t length;
    uint32_t err;
    if (blockIdx.x >= turning) {
        store_values<T, C>(a, blockIdx.x - turning, tiles, lds);
        return;
    }

    // rotate q and k of R rows
    float2 *cs = (float2 *)lds;
    const int32_t pairs = a.rot_dim / 2;
    const uint32_t groups = (uint32_t)(g.rows + R - 1) / R;
    const int32_t b = blockIdx.x / groups, t0 = blockIdx.x % groups * R;
    const int32_t n = block_rows(g, b, length, err);
    if (t0 >= n) {
        if (err && t0 == 0 && tid == 0)
            atomicOr(g.err, err);
        return;
    }
    const int32_t live = n - t0 < R ? n - t0 : R;
    int32_t *pages = (int32_t *)(cs + R * kMaxPairs);
    // units of a head: with the half layout a word of the first half and its
    // partner are one, else every word is one
    const int32_t twos = a.interleaved ? 0 : pairs / 8;
    const uint32_t units = dim / 8 - twos;
    const uint32_t q_heads = a.q ? g.q_heads : 0, heads = q_heads + g.kv_heads;
    const uint32_t all = live * heads * units;
    struct Unit {
        Eight<T> u, v;
        uint32_t unit, h, t;
    };
    const auto fetch = [&](uint32_t i) {
        Unit x;
        x.unit = i % units;
        const uint32_t hr = i / units;
        x.h = hr % heads;
        x.t = hr / heads;
        const int64_t r = (int64_t)b * g.rows + t0 + x.t;
        const T *from = x.h < q_heads ? (const T *)a.q + r * a.q_stride + (int64_t)x.h * dim
                                      : (const T *)a.k + r * a.kv_stride +
                                            (int64_t)(x.h - q_heads) * dim;
        const bool two = x.unit < (uint32_t)twos;
        const T *p = from + (two ? x.unit : x.unit + twos) * 8;
        x.u = load8(p);
        x.v = x.u;
        if (two)
            x.v = load8(p + pairs);
        return x;
    };
    // Few rows: the first words are on their way before the angles (13.6 ->
    // 11.1 us for 64 blocks of 16 rows). Many rows hide that latency in each
    // other and would only lose wavefronts to the registers (326 -> 338 us for
    // 65,536 rows).
    constexpr bool kAhead = R == 1;
    Unit next{};
    if (kAhead && (uint32_t)tid < all)
        next = fetch(tid);
    if (tid >= kThreads - live) {
        const int32_t t = tid - (kThreads - live);
        pages[t] = page_of(g, b, length - 1 + t0 + t);
        if (pages[t] < 0)
            atomicOr(g.err, (uint32_t)kErrPage);
    }
    for (int32_t i = tid; i < live * pairs; i += kThreads) {
        float c, s;
        turn(a.turns[i % pairs], length - 1 + t0 + i / pairs, a.magnitude, c, s);
        cs[i] = float2{c, s};
    }
    __syncthreads();
    for (uint32_t i = tid; i < all; i += kThreads) {
        const Unit x = kAhead ? next : fetch(i);
        if (kAhead && i + kThreads < all)
            next = fetch(i + kThreads);
        const int64_t r = (int64_t)b * g.rows + t0 + x.t;
        const float2 *w = cs + x.t * pairs;
        const bool two = x.unit < (uint32_t)twos;
        const int32_t d = (two ? x.unit : x.unit + twos) * 8;
        float y[8], z[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            y[k] = to_f32(x.u.x[k]);
        if (two) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float e = y[k], f = to_f32(x.v.x[k]);
                const float2 m = w[d + k];
                y[k] = e * m.x - f * m.y;
                z[k] = e * m.y + f * m.x;
            }
        } else if (d < a.rot_dim) {
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const float e = y[k], f = y[k + 1];
                const float2 m = w[(d + k) / 2];
                y[k] = e * m.x - f * m.y;
                y[k + 1] = e * m.y + f * m.x;
            }
        }
        if (x.h < q_heads) {
            T *out = (T *)a.out_q + (r * g.q_heads + x.h) * dim + d;
            store8<T>(out, y);
            if (two)
                store8<T>(out + pairs, z);
            continue;
        }
        const int32_t page = pages[x.t], h = x.h - q_heads;
        if (page < 0)
            continue;
        if (g.k_scale) {
            const float scale = g.k_scale[h];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                y[k] /= scale;
                z[k] /= scale;
            }
        }
        C *out = (C *)a.k_cache +
                 (((int64_t)page * g.kv_heads + h) * tokens +
                  ((length - 1 + t0 + (int32_t)x.t) & (tokens - 1))) * dim + d;
        store8<C>(out, y);
        if (two)
            store8<C>(out + pairs, z);
    }
}

// Any alignment and any part of a head: one workgroup per row, an element at
// a time.
template <typename T, typename C>
__global__ __launch_bounds__(kThreads) void append_elements(KvAppendArgs a)
{
    const BlockArgs &g = a.blk;
    const int32_t t = (int32_t)(blockIdx.x % (uint32_t)g.rows);
    const int32_t b = (int32_t)(blockIdx.x / (uint32_t)g.rows);
    int32_t length;
    uint32_t err;
    const int32_t n = block_rows(g, b, length, err);
    if (t >= n) {
        if (err && t == 0 && threadIdx.x == 0)
            atomicOr(g.err, err);
        return;
    }
    const int32_t p = length - 1 + t;
    const int32_t page = page_of(g, b, p);
    if (page < 0 && threadIdx.x == 0)
        atomicOr(g.err, (uint32_t)kErrPage);
    const int32_t dim = g.head_dim, half = a.rot_dim / 2, tokens = 1 << g.page_shift;
    const int32_t slot = p & (tokens - 1);
    const int64_t r = (int64_t)b * g.rows + t;
    const int32_t heads = a.q ? g.q_heads : 0;
    // (both elements of a pair go through one thread: q may be rotated in place)
    const int32_t units = dim - half;
    for (int32_t i = threadIdx.x; i < (heads + g.kv_heads) * units; i += blockDim.x) {
        const int32_t h = i / units, e = i % units;
        const bool is_q = h < heads, two = e < half;
        const T *x = is_q ? (const T *)a.q + r * a.q_stride + (int64_t)h * dim
                          : (const T *)a.k + r * a.kv_stride + (int64_t)(h - heads) * dim;
        const int32_t d = two ? (a.interleaved ? 2 * e : e) : e + half;
        const int32_t d2 = two ? (a.interleaved ? d + 1 : d + half) : d;
        float y = to_f32(x[d]), z = to_f32(x[d2]);
        if (two) {
            float c, s;
            turn(a.turns[e], p, a.magnitude, c, s);
            const float y0 = y;
            y = y0 * c - z * s;
            z = y0 * s + z * c;
        }
        if (is_q) {
            T *out = (T *)a.out_q + (r * g.q_heads + h) * dim;
            out[d] = from_f32<T>(y);
            if (two)
                out[d2] = from_f32<T>(z);
        } else if (page >= 0) {
            const float scale = g.k_scale ? g.k_scale[h - heads] : 1.0f;
            C *out = (C *)a.k_cache +
                     (((int64_t)page * g.kv_heads + h - heads) * tokens + slot) * dim;
            out[d] = from_f32<C>(y / scale);
            if (two)
                out[d2] = from_f32<C>(z / scale);
        }
    }
    if (page < 0)
        return;
    for (int32_t i = threadIdx.x; i < g.kv_heads * dim; i += blockDim.x) {
        const float scale = g.v_scale ? g.v_scale[i / dim] : 1.0f;
        ((C *)a.v_cache)[((int64_t)page * g.kv_heads * dim + i) * tokens + slot] =
            from_f32<C>(to_f32(((const T *)a.v)[r * a.kv_stride + i]) / scale);
    }
}

template <typename T, typename C>
hipError_t launch_cells(const KvAppendArgs &a, hipStream_t s)
{
    const BlockArgs &g = a.blk;
    const int64_t rows = (int64_t)g.batch * g.rows;
    const bool words = !(((uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.out_q) &
                         15u) &&
                       !((a.q ? a.q_stride : 0) & 7) && !(a.kv_stride & 7) &&
                       a.rot_dim % (a.interleaved ? 8 : 16) == 0;
    if (!words) {
        if (!fits_grid(rows, kThreads))
            return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((append_elements<T, C>), dim3((uint32_t)rows), dim3(kThreads), 0, s, a);
        return hipGetLastError();
    }
    // 4 rows a workgroup share its start once there are enough of them. Measured,
    // 1 and 4 rows (rows of the padded blocks, 16 a request; q, k and v heads):
    // 512 rows of 64 + 8 + 8: 8.8 and 11.9 us, of 32 + 8 + 8: 7.7 and 8.0; 1,024:
    // 13.6 and 13.7, 11.5 and 10.5; 1,536: 17.2 and 15.7, 14.8 and 14.5; 2,048: 21.0
    // and 18.9, 17.8 and 17.2. One long block: 1,024 rows of 64 + 8 + 8 11.3 and 13.4,
    // 1,536 15.1 and 15.4, 2,048 16.9 and 16.9; of 32 + 8 + 8 9.6 and 8.3, 12.4 and
    // 10.3, 13.8 and 11.2.
    const int R = rows >= kManyRows ? 4 : 1;
    const int64_t turning = (int64_t)g.batch * ((g.rows + R - 1) / R);
    const int64_t tiles = (g.rows + kSpan - 2) / kSpan + 1;
    const int64_t storing = (int64_t)g.batch * g.kv_heads * tiles;
    if (!fits_grid(turning + storing, kThreads))
        return hipErrorInvalidConfiguration;
    const size_t turn_lds = (size_t)R * (kMaxPairs * sizeof(float2) + sizeof(int32_t));
    const size_t tile_lds = (size_t)kSpan * (g.head_dim + kPad) * sizeof(T);
    const size_t lds = turn_lds > tile_lds ? turn_lds : tile_lds;
    const dim3 grid((uint32_t)(turning + storing));
    if (R == 4)
        hipLaunchKernelGGL((append_words<T, C, 4>), grid, dim3(kThreads), lds, s, a,
                           (uint32_t)turning, (uint32_t)tiles);
    else
        hipLaunchKernelGGL((append_words<T, C, 1>), grid, dim3(kThreads), lds, s, a,
                           (uint32_t)turning, (uint32_t)tiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s)
{
    const bool wide = a.blk.cache_dtype != PLD_E4M3;
    if (a.blk.dtype == PLD_BF16)
        return wide ? launch_cells<__bf16, __bf16>(a, s) : launch_cells<__bf16, E4m3>(a, s);
    return wide ? launch_cells<_Float16, _Float16>(a, s) : launch_cells<_Float16, E4m3>(a, s);
}

}  // namespace pld
