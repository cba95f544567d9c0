// Attention of the verify block's rows over the paged cache, for gfx950
// (MI355X).

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pld_target_device.h"

namespace pld {

namespace {

constexpr int kWave = 64;

// One wavefront per (request, row, query head): 64 positions at a time, one
// per lane for the scores and one dim per lane for the sum.
template <typename T, typename C, int D>
__global__ __launch_bounds__(kWave) void attend_kernel(AttendArgs a)
{
    const BlockArgs &g = a.blk;
    const int32_t lane = threadIdx.x;
    const int32_t h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    int32_t length;
    uint32_t err;
    const int32_t n = block_rows(g, b, length, err);
    if (n >= 0 && t >= n)
        return;
    if (err && h == 0 && t == 0 && lane == 0)
        atomicOr(g.err, err);
    const int64_t r = (int64_t)b * g.rows + t;
    T *out = (T *)a.out + (r * g.q_heads + h) * D;
    float *lse = a.out_lse ? a.out_lse + r * g.q_heads + h : nullptr;
    const int32_t kvh = h / (g.q_heads / g.kv_heads);
    const int32_t tokens = 1 << g.page_shift;
    const int32_t p = length - 1 + t;
    const int32_t lo = a.window && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    const T *q = (const T *)a.q + r * a.q_stride + (int64_t)h * D;
    const float ks = g.k_scale ? g.k_scale[kvh] : 1.0f, vs = g.v_scale ? g.v_scale[kvh] : 1.0f;
    float m = -INFINITY, l = 0.0f, o[D / 32] = {};
    bool bad = n < 0;
    for (int32_t j0 = bad ? p + 1 : lo / kWave * kWave; j0 <= p; j0 += kWave) {
        const int32_t j = j0 + lane;
        float s = -INFINITY;
        if (j >= lo && j <= p) {
            const int32_t page = page_of(g, b, j);
            if (page < 0) {
                bad = true;
            } else {
                const C *k = (const C *)a.k_cache +
                             (((int64_t)page * g.kv_heads + kvh) * tokens + (j & (tokens - 1))) * D;
                s = 0.0f;
                for (int i = 0; i < D; ++i)
                    s += to_f32(q[i]) * to_f32(k[i]);
                s *= a.scale * ks;
            }
        }
        if (__any(bad))
            break;
        float mt = s;
        for (int i = kWave / 2; i; i >>= 1)
            mt = fmaxf(mt, __shfl_xor(mt, i));
        mt = fmaxf(m, mt);
        const float base = mt == -INFINITY ? 0.0f : mt;
        const float e = __expf(s - base), old = __expf(m - base);
        float sum = e;
        for (int i = kWave / 2; i; i >>= 1)
            sum += __shfl_xor(sum, i);
        l = l * old + sum;
        m = mt;
        for (int i = 0; i < D / 32; ++i)
            o[i] *= old;
        for (int u = 0; u < kWave; ++u) {
            const int32_t ju = j0 + u;
            if (ju < lo || ju > p)
                continue;
            const float pu = __shfl(e, u);
            const int32_t page = page_of(g, b, ju);
            const C *v = (const C *)a.v_cache +
                         (((int64_t)page * g.kv_heads + kvh) * D) * tokens + (ju & (tokens - 1));
            for (int i = 0; i < D / 32; ++i) {
                const int d = lane + i * kWave;
                if (d < D)
                    o[i] += pu * to_f32(v[(int64_t)d * tokens]);
            }
        }
    }
    if (__any(bad)) {
        if (n >= 0 && lane == 0)
            atomicOr(g.err, (uint32_t)kErrPage);
        l = NAN;
    }
    for (int i = 0; i < D / 32; ++i) {
        const int d = lane + i * kWave;
        if (d < D)
            out[d] = from_f32<T>(o[i] * vs / l);
    }
    if (lse && lane == 0)
        *lse = m + __logf(l);
}

template <typename T, typename C>
hipError_t launch_typed(const AttendArgs &a, hipStream_t s)
{
    const dim3 grid(a.blk.q_heads, a.blk.rows, a.blk.batch), block(kWave);
    switch (a.blk.head_dim) {
    case 64: hipLaunchKernelGGL((attend_kernel<T, C, 64>), grid, block, 0, s, a); break;
    case 96: hipLaunchKernelGGL((attend_kernel<T, C, 96>), grid, block, 0, s, a); break;
    case 128: hipLaunchKernelGGL((attend_kernel<T, C, 128>), grid, block, 0, s, a); break;
    case 192: hipLaunchKernelGGL((attend_kernel<T, C, 192>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((attend_kernel<T, C, 256>), grid, block, 0, s, a); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attend(const AttendArgs &a, hipStream_t s)
{
    const bool wide = a.blk.cache_dtype != PLD_E4M3;
    if (a.blk.dtype == PLD_BF16)
        return wide ? launch_typed<__bf16, __bf16>(a, s) : launch_typed<__bf16, E4m3>(a, s);
    return wide ? launch_typed<_Float16, _Float16>(a, s) : launch_typed<_Float16, E4m3>(a, s);
}

}  // namespace pld
