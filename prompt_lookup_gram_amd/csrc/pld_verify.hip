// Verification of drafted tokens against the target model's logits, for
// gfx950 (MI355X).

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pld_target_device.h"

namespace pld {

namespace {

constexpr int kWave = 64;
constexpr int kPiece = 4096;      // logits of a row per wavefront
constexpr int kFinish = 1024;     // threads of the finishing workgroup

// Statistics of a piece of a row: the largest logit, its lowest index, and
// the sum of exp((z - top) / T). A NaN or +inf in the piece makes the sum NaN.
struct Piece {
    float top;
    float sum;
    int32_t arg;
};

__device__ __forceinline__ float temperature(const VerifyArgs &a, int32_t b)
{
    return a.temperature ? a.temperature[b] : 1.0f;
}

// One wavefront per piece of a row.
template <typename T>
__global__ __launch_bounds__(kWave) void stats_kernel(VerifyArgs a)
{
    const int32_t b = blockIdx.z, t = blockIdx.y;
    if (t > a.draft_len[b])
        return;
    const float temp = temperature(a, b);
    const float c = 1.0f / (temp > 0.0f ? temp : 1.0f);
    const T *z = (const T *)a.logits + ((int64_t)b * a.rows + t) * a.stride;
    const int32_t lo = blockIdx.x * kPiece;
    const int32_t hi = lo + kPiece < a.vocab ? lo + kPiece : a.vocab;
    float top = -INFINITY;
    int32_t arg = 0x7fffffff;
    for (int32_t i = lo + threadIdx.x; i < hi; i += kWave) {
        const float x = to_f32(z[i]);
        if (x > top) {
            top = x;
            arg = i;
        }
    }
    for (int i = kWave / 2; i; i >>= 1) {
        const float x = __shfl_xor(top, i);
        const int32_t k = __shfl_xor(arg, i);
        if (x > top || (x == top && k < arg)) {
            top = x;
            arg = k;
        }
    }
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (int32_t i = lo + threadIdx.x; i < hi; i += kWave)
        sum += __expf((to_f32(z[i]) - base) * c);
    for (int i = kWave / 2; i; i >>= 1)
        sum += __shfl_xor(sum, i);
    if (threadIdx.x == 0)
        ((Piece *)a.stats)[((int64_t)b * a.rows + t) * gridDim.x + blockIdx.x] =
            Piece{top, sum, arg};
}

// Sum over the workgroup, the same on every thread.
__device__ double block_sum(double x, double *lds)
{
    for (int i = kWave / 2; i; i >>= 1)
        x += __shfl_xor(x, i);
    __syncthreads();
    if (threadIdx.x % kWave == 0)
        lds[threadIdx.x / kWave] = x;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < kFinish / kWave; ++w)
        s += lds[w];
    return s;
}

// One workgroup per request: accepts its draft row by row, then draws.
template <typename T>
__global__ __launch_bounds__(kFinish) void finish_kernel(VerifyArgs a, int32_t pieces)
{
    __shared__ double lds[kFinish / kWave];
    __shared__ double run[kFinish];
    __shared__ int32_t pick, last;
    const int32_t b = blockIdx.x, tid = threadIdx.x, v = a.vocab;
    const int32_t d = a.draft_len[b];
    const float tf = temperature(a, b);
    const bool greedy = tf == 0.0f;
    const double inv = greedy ? 1.0 : 1.0 / (double)tf;
    const float *u = a.uniform + (int64_t)b * a.rows;
    const int32_t *x = a.draft + (int64_t)b * (a.rows - 1);
    bool bad = d < -1 || d >= a.rows || !(tf >= 0.0f) || tf == INFINITY;
    if (!bad && d >= 0) {
        for (int32_t t = 0; t < d; ++t)
            bad |= x[t] < 0 || x[t] >= v || (!greedy && !(u[t] >= 0.0f && u[t] < 1.0f));
        bad |= !greedy && !(u[a.rows - 1] >= 0.0f && u[a.rows - 1] < 1.0f);
    }
    int32_t accepted = 0, token = -1;
    for (int32_t t = 0; !bad && t <= d; ++t) {
        const T *z = (const T *)a.logits + ((int64_t)b * a.rows + t) * a.stride;
        const Piece *pc = (const Piece *)a.stats + ((int64_t)b * a.rows + t) * pieces;
        float top = -INFINITY;
        int32_t arg = 0;
        bool nan = false;
        for (int32_t i = 0; i < pieces; ++i) {
            nan |= !(pc[i].sum >= 0.0f);
            if (pc[i].top > top) {
                top = pc[i].top;
                arg = pc[i].arg;
            }
        }
        if (nan || top == -INFINITY || top == INFINITY) {
            bad = true;
            break;
        }
        double part = 0.0;
        for (int32_t i = tid; i < v; i += kFinish)
            part += exp(((double)to_f32(z[i]) - top) * inv);
        const double total = block_sum(part, lds);
        bool take = false;
        const bool claimed = t < d && t < a.head &&
                             !(a.src && t < 64 && ((a.src[b] >> t) & 1));
        const float *q = claimed ? a.probs + ((int64_t)b * a.head + t) * v : nullptr;
        if (t < d) {
            const double p = exp(((double)to_f32(z[x[t]]) - top) * inv) / total;
            take = greedy ? x[t] == arg : (double)u[t] * (q ? (double)q[x[t]] : 1.0) < p;
        }
        if (take) {
            token = x[t];
        } else if (greedy) {
            token = arg;
        } else {
            // weights of the draw: mode 0 the row's own, 1 without x_t, 2 the
            // excess over q
            int mode = t == d ? 0 : (q ? 2 : 1);
            const auto weight = [&](int32_t i) {
                const double w = exp(((double)to_f32(z[i]) - top) * inv);
                if (mode == 1)
                    return i == x[t] ? 0.0 : w;
                const double e = w - (mode == 2 ? (double)q[i] * total : 0.0);
                return e > 0.0 ? e : 0.0;
            };
            const int32_t per = (v + kFinish - 1) / kFinish;
            const int32_t lo = tid * per < v ? tid * per : v;
            const int32_t hi = lo + per < v ? lo + per : v;
            double all = 0.0;
            for (; mode >= 0; mode = mode == 2 ? 0 : -1) {
                part = 0.0;
                for (int32_t i = lo; i < hi; ++i)
                    part += weight(i);
                all = block_sum(part, lds);
                if (all > 0.0 || mode == 0)
                    break;
            }
            if (mode < 0)
                mode = 0;
            run[tid] = part;
            if (tid == 0)
                pick = last = -1;
            __syncthreads();
            double before = 0.0;
            for (int w = 0; w < tid; ++w)
                before += run[w];
            const double goal = (double)u[a.rows - 1] * all;
            for (int32_t i = lo; i < hi; ++i) {
                const double w = weight(i);
                if (w > 0.0) {
                    if (before + w > goal) {
                        if (before <= goal)
                            atomicMax(&pick, i);
                    }
                    before += w;
                    atomicMax(&last, i);
                }
            }
            __syncthreads();
            // the running sum's last rounding may end just at the goal
            token = pick >= 0 ? pick : last;
        }
        if (tid == 0) {
            a.out_tokens[(int64_t)b * a.rows + t] = token;
            if (a.out_logprobs)
                a.out_logprobs[(int64_t)b * a.rows + t] =
                    (float)(((double)to_f32(z[token]) - top) * inv - log(total));
        }
        accepted = t;
        if (!take)
            break;
    }
    if (bad && tid == 0)
        atomicOr(a.err, (uint32_t)kErrBlock);
    const int32_t count = bad || d < 0 ? 0 : accepted + 1;
    for (int32_t t = count + tid; t < a.rows; t += kFinish) {
        a.out_tokens[(int64_t)b * a.rows + t] = -1;
        if (a.out_logprobs)
            a.out_logprobs[(int64_t)b * a.rows + t] = 0.0f;
    }
    if (tid == 0) {
        a.out_accepted[b] = count > 0 ? accepted : 0;
        a.out_counts[b] = count;
    }
}

int32_t pieces_of(int32_t vocab) { return (vocab + kPiece - 1) / kPiece; }

template <typename T>
hipError_t launch_typed(const VerifyArgs &a, hipStream_t s)
{
    const int32_t pieces = pieces_of(a.vocab);
    hipLaunchKernelGGL((stats_kernel<T>), dim3(pieces, a.rows, a.batch), dim3(kWave), 0, s, a);
    hipLaunchKernelGGL((finish_kernel<T>), dim3(a.batch), dim3(kFinish), 0, s, a, pieces);
    return hipGetLastError();
}

}  // namespace

size_t verify_workspace(int32_t batch, int32_t rows, int32_t vocab)
{
    return (size_t)batch * rows * pieces_of(vocab) * sizeof(Piece);
}

hipError_t launch_verify(const VerifyArgs &a, hipStream_t s)
{
    switch (a.dtype) {
    case PLD_F32: return launch_typed<float>(a, s);
    case PLD_F16: return launch_typed<_Float16>(a, s);
    default: return launch_typed<__bf16>(a, s);
    }
}

}  // namespace pld
