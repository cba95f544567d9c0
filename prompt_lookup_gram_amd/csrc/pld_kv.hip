// Rotary positions and the paged cache's writer, for gfx950 (MI355X).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pld_target_device.h"

namespace pld {

namespace {

// cos and sin of the angle `turns` per position reaches at position p: the
// angle is reduced to one turn in 64 bits (at position 262,144 a 32-bit
// product would be off by 2^-6 radians), the functions are 32-bit.
__device__ __forceinline__ void turn(double turns, int32_t p, float &c, float &s)
{
    const double x = turns * p;
    sincospif((float)(2.0 * (x - rint(x))), &s, &c);
}

// One workgroup per row of a block.
template <typename T, typename C>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a)
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
    for (int32_t i = threadIdx.x; i < (heads + g.kv_heads) * dim; i += blockDim.x) {
        const int32_t h = i / dim, d = i % dim;
        const bool is_q = h < heads;
        const T *x = is_q ? (const T *)a.q + r * a.q_stride + (int64_t)h * dim
                          : (const T *)a.k + r * a.kv_stride + (int64_t)(h - heads) * dim;
        float y = to_f32(x[d]);
        if (d < a.rot_dim) {
            const int32_t i2 = a.interleaved ? d / 2 : (d < half ? d : d - half);
            const bool first = a.interleaved ? !(d & 1) : d < half;
            const int32_t other = a.interleaved ? (d ^ 1) : (first ? d + half : d - half);
            float c, s;
            turn(a.turns[i2], p, c, s);
            const float z = to_f32(x[other]);
            y = (first ? y * c - z * s : z * s + y * c) * a.magnitude;
        }
        if (is_q) {
            ((T *)a.out_q)[r * g.q_heads * dim + (int64_t)h * dim + d] = from_f32<T>(y);
        } else if (page >= 0) {
            const float scale = g.k_scale ? g.k_scale[h - heads] : 1.0f;
            ((C *)a.k_cache)[(((int64_t)page * g.kv_heads + h - heads) * tokens + slot) * dim + d] =
                from_f32<C>(y / scale);
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

template <typename T>
void launch_typed(const KvAppendArgs &a, hipStream_t s)
{
    const dim3 grid((uint32_t)a.blk.batch * (uint32_t)a.blk.rows);
    if (a.blk.cache_dtype == PLD_E4M3)
        hipLaunchKernelGGL((kv_append_kernel<T, E4m3>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((kv_append_kernel<T, T>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s)
{
    if (a.blk.dtype == PLD_BF16)
        launch_typed<__bf16>(a, s);
    else
        launch_typed<_Float16>(a, s);
    return hipGetLastError();
}

}  // namespace pld
