// Device helpers that the verifications of a chain and of a tree share: the
// workspace, what crosses workgroups, and a row's sum in more bits.
#pragma once

#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "pld_target_device.h"

namespace pld {

namespace {

constexpr int kWave = 64;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMinUnit = 512;               // logits whose weights are summed together
constexpr int32_t kNever = 0x7f7f7f7f;      // `stop` before a refusal
constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLog2e64 = 1.4426950408889634074;
constexpr double kClear = 1.0 / (1 << 17);  // relative distances that the 32-bit sum
constexpr double kClearer = 1.0 / (1 << 22);  // and the one after it decide

// A piece of a row: the largest logit, the sum of exp((z - top) / T) (NaN
// when it holds NaN or +inf), and the lowest index of the largest (greedy).
struct Piece {
    unsigned long long top_sum;
    unsigned long long arg;
};

// A row, decided.
struct Row {
    double total;
    float top;
    float logp;      // of the draft token
    int32_t arg;     // greedy
    int32_t verdict;
    int32_t pad[2];
};

// The workspace, laid out for `rows` rows and `vocab` logits.
struct Space {
    Piece *pieces;      // [batch * rows][pieces]
    Row *rows;          // [batch * rows]
    double *weights;    // [batch][units]: sums of a row's weights
    double *excess;     // [batch][units]: the same over q
    int32_t *arrived;   // [batch * rows], 0 between calls
    int32_t *drawn;     // [batch], 0 between calls
    int32_t *stop;      // [batch], kNever between calls
};

constexpr int kMinPiece = 2048;
constexpr int64_t kManyPieces = 32;

__host__ __device__ int64_t pieces_of(int32_t vocab, int piece)
{
    return ((int64_t)vocab + piece - 1) / piece;
}

// Offsets by the context's sizes, so that every call of a context agrees.
__host__ __device__ Space space_of(char *p, int64_t batch, int64_t rows, int32_t vocab,
                                   size_t *size)
{
    Space s;
    char *const from = p;
    s.pieces = (Piece *)p;
    p += batch * rows * pieces_of(vocab, kMinPiece) * sizeof(Piece);
    s.rows = (Row *)p;
    p += batch * rows * sizeof(Row);
    s.weights = (double *)p;
    p += batch * pieces_of(vocab, kMinUnit) * sizeof(double);
    s.excess = (double *)p;
    p += batch * pieces_of(vocab, kMinUnit) * sizeof(double);
    s.arrived = (int32_t *)p;
    p += batch * rows * sizeof(int32_t);
    s.drawn = (int32_t *)p;
    p += batch * sizeof(int32_t);
    s.stop = (int32_t *)p;
    p += batch * sizeof(int32_t);
    if (size)
        *size = (size_t)(p - from);
    return s;
}

template <typename X>
__device__ __forceinline__ X peek(const X *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename X>
__device__ __forceinline__ void poke(X *p, X v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Counts this workgroup in, its stores before it complete; thread 0 only.
__device__ __forceinline__ int32_t arrive(int32_t *counter)
{
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    return __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ float temperature(const VerifyArgs &a, int32_t b)
{
    return a.temperature ? a.temperature[b] : 1.0f;
}

__device__ __forceinline__ float wave_max(float x)
{
    for (int i = kWave / 2; i; i >>= 1)
        x = fmaxf(x, __shfl_xor(x, i));
    return x;
}
template <typename X>
__device__ __forceinline__ X wave_sum(X x)
{
    for (int i = kWave / 2; i; i >>= 1)
        x += __shfl_xor(x, i);
    return x;
}

// Sum over the workgroup, the same on every thread.
__device__ __forceinline__ double block_sum(double x, double *lds)
{
    x = wave_sum(x);
    __syncthreads();
    if (threadIdx.x % kWave == 0)
        lds[threadIdx.x / kWave] = x;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < (int)blockDim.x / kWave; ++w)
        s += lds[w];
    return s;
}

// 16 bytes of logits at any element's address.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Word {
    T x[16 / sizeof(T)];
};

// sum exp((z - m) inv) over a row by one wavefront, to 2^-22: 2^y with y in 64
// bits, its whole part split off before the 32-bit function.
template <typename T>
__device__ __forceinline__ double sum_again(const T *z, int32_t vocab, float m, double inv, int lane)
{
    constexpr int N = 16 / sizeof(T), kDeep = 4;
    const double c = inv * kLog2e64;
    double sum = 0.0;
    const auto add = [&](float x) {
        const double y = ((double)x - m) * c, n = rint(y);
        // (below 2^-149 the weight is 0, the whole part may be -infinity)
        if (n > -150.0)
            sum += (double)ldexpf(__builtin_amdgcn_exp2f((float)(y - n)), (int)n);
    };
    int32_t i = lane * N;
    for (; i <= vocab - (kDeep - 1) * kWave * N - N; i += kDeep * kWave * N) {
        Word<T> w[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            w[k] = *(const Word<T> *)(z + i + k * kWave * N);
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e)
                add(to_f32(w[k].x[e]));
    }
    for (; i < vocab; i += kWave * N)
        for (int e = 0; e < N && i + e < vocab; ++e)
            add(to_f32(z[i + e]));
    return wave_sum(sum);
}

}  // namespace

}  // namespace pld
