// Verification of drafted tokens against the target model's logits, for
// gfx950 (MI355X).
//
// Mathematics. For every row t of a block: top_t = max z, Z_t = sum exp((z -
// top_t) / T) in one read of the row; the draft token is accepted when u q <
// exp((z_x - top_t) / T) / Z_t. The row after the accepted ones is read once
// more, in 64 bits, for the draw: running sums of weights over pieces, then
// inside the piece that holds u times the total.
//
// Bound by reading the rows (2 or 4 bytes a logit, 7.5 vector operations at
// 16 bits, about the two's balance). Three things follow:
//  - a piece of a row lives in one workgroup's registers between the maximum
//    and the sum, so it is read once;
//  - rows are dispatched in the order of t, and the workgroup that completes
//    a row decides it; rows after one that is refused are skipped as soon as
//    that is known (`stop`). What is skipped never changes a result: only
//    rows up to the first refusal are looked at;
//  - the 32-bit sum decides only where it is clear. Its relative error is
//    below 48 * 2^-23: an argument y is off by 1.5 * 2^-23 |y|, which the
//    softmax weighs to at most 1.5 ln V * 2^-23 = 25 * 2^-23 for V <= 2^24, the
//    function by 2^-23, 40 additions by 20 * 2^-23. Within 2^-17 of the edge (one decision in 65,000) the deciding
//    wavefront sums the row again with 64-bit arguments and sums, which
//    leaves the function's 2^-23 (75 us for 151,936 logits), and within 2^-22
//    with 64-bit exponentials as well (430 us).
// Numbers that cross workgroups do so in relaxed agent-scope atomics, each
// performed at the point of coherence; a workgroup waits for its stores to
// complete before it counts itself in, so who counts last reads them all.

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

enum : int32_t { kAccept = 0, kRefuse = 1, kBad = 2 };

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

// Whether position t of request b has drafter probabilities.
__device__ __forceinline__ const float *claim_of(const VerifyArgs &a, int32_t b, int32_t t,
                                                 int32_t d)
{
    if (t >= d || t >= a.head || (a.src && t < 64 && ((a.src[b] >> t) & 1)))
        return nullptr;
    return a.probs + ((int64_t)b * a.head + t) * a.vocab;
}

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

// One workgroup per piece of a row, W 16-byte words a thread.
// Measured: 64 requests of up to 16 draft tokens, 151,936 bf16 logits a row:
// 33 us, 121 MB read where 57 are up to the refusals; one request of 17 rows of
// 32,000: 7.1 us, the chain of its round trips.
// (8 wavefronts a SIMD: the rare second sum must not cost the first its
// registers)
template <typename T, int W>
__global__ __launch_bounds__(kThreads, 8) void stats_kernel(VerifyArgs a, Space sp, uint32_t pieces)
{
    constexpr int N = 16 / sizeof(T);
    constexpr int kPiece = W * N * kThreads;
    __shared__ float lds_max[kWaves], lds_sum[kWaves];
    __shared__ int32_t lds_arg[kWaves], lds_stop;
    const int32_t piece = blockIdx.x % pieces, tid = threadIdx.x;
    const uint32_t order = blockIdx.x / pieces;
    const int32_t b = order % (uint32_t)a.batch, t = order / (uint32_t)a.batch;
    const int wave = tid / kWave, lane = tid % kWave;
    const int32_t d = a.draft_len[b];
    if (t > d || d >= a.rows)
        return;
    // (`stop` may change between two reads: one decides for all wavefronts)
    if (tid == 0)
        lds_stop = peek(sp.stop + b);
    __syncthreads();
    if (lds_stop < t)
        return;
    const T *z = (const T *)a.logits + ((int64_t)b * a.rows + t) * a.stride;
    const float tf = temperature(a, b);
    const bool greedy = tf == 0.0f;
    const float c = kLog2e / (greedy ? 1.0f : tf);

    // what deciding the row takes, on its way with the row
    const int32_t token = t < d ? a.draft[(int64_t)b * (a.rows - 1) + t] : -1;
    const bool known = token >= 0 && token < a.vocab;
    const float *q = claim_of(a, b, t, d);
    const float claim = q && known ? q[token] : 1.0f;
    const float z_token = known ? to_f32(z[token]) : 0.0f;
    const float u = a.uniform[(int64_t)b * a.rows + t];

    float x[W * N];
    float top = -INFINITY;
    const int32_t lo = piece * kPiece + tid * N;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int32_t i = lo + w * (kThreads * N);
        if (i <= a.vocab - N) {
            const Word<T> y = *(const Word<T> *)(z + i);
#pragma unroll
            for (int k = 0; k < N; ++k)
                x[w * N + k] = to_f32(y.x[k]);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
                x[w * N + k] = i + k < a.vocab ? to_f32(z[i + k]) : -INFINITY;
        }
    }
#pragma unroll
    for (int k = 0; k < W * N; ++k)
        top = fmaxf(top, x[k]);
    top = wave_max(top);
    if (lane == 0)
        lds_max[wave] = top;
    __syncthreads();
    top = lds_max[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        top = fmaxf(top, lds_max[w]);
    // (without a finite logit the sum is 0, or NaN with a NaN.) One operation a
    // logit where what rounding takes off the common exponent is small enough
    // to be put back into the sum; far logits take two.
    float base = top * c, rest = 0.0f, sum = 0.0f;
    if (fabsf(base) < 1048576.0f) {
        rest = fmaf(top, c, -base);
#pragma unroll
        for (int k = 0; k < W * N; ++k)
            sum += __builtin_amdgcn_exp2f(fmaf(x[k], c, -base));
    } else {
        base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int k = 0; k < W * N; ++k)
            sum += __builtin_amdgcn_exp2f((x[k] - base) * c);
    }
    sum = wave_sum(sum);
    int32_t arg = 0x7fffffff;
    if (greedy) {
#pragma unroll
        for (int k = W * N - 1; k >= 0; --k)
            if (x[k] == top)
                arg = lo + k / N * (kThreads * N) + k % N;
        for (int i = kWave / 2; i; i >>= 1) {
            const int32_t y = __shfl_xor(arg, i);
            arg = y < arg ? y : arg;
        }
    }
    if (lane == 0) {
        lds_sum[wave] = sum;
        lds_arg[wave] = arg;
    }
    __syncthreads();
    if (wave > 0)
        return;  // one wavefront counts the piece in, and decides if it is the last
    const int64_t r = (int64_t)b * a.rows + t;
    Piece *const mine = sp.pieces + r * pieces;
    int32_t count = 0;
    if (lane == 0) {
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            sum += lds_sum[w];
            arg = lds_arg[w] < arg ? lds_arg[w] : arg;
        }
        sum *= __builtin_amdgcn_exp2f(-rest);
        poke(&mine[piece].top_sum,
             (unsigned long long)__float_as_uint(top) << 32 | __float_as_uint(sum));
        if (greedy)
            poke(&mine[piece].arg, (unsigned long long)(uint32_t)arg);
        count = arrive(sp.arrived + r);
    }
    if (__builtin_amdgcn_readfirstlane(count) != (int32_t)pieces - 1)
        return;

    // this wavefront completes the row: join the pieces and decide
    const double inv = greedy ? 1.0 : 1.0 / (double)tf;
    const double weight = greedy ? 0.0 : (double)u * (double)claim;
    float m = -INFINITY;
    for (uint32_t i = lane; i < pieces; i += kWave)
        m = fmaxf(m, __uint_as_float((uint32_t)(peek(&mine[i].top_sum) >> 32)));
    m = wave_max(m);
    int32_t best = 0x7fffffff;
    double total = 0.0;
    for (uint32_t i = lane; i < pieces; i += kWave) {
        const unsigned long long v = peek(&mine[i].top_sum);
        const float pt = __uint_as_float((uint32_t)(v >> 32));
        const float ps = __uint_as_float((uint32_t)v);
        total += pt == -INFINITY ? (double)ps : (double)ps * exp(((double)pt - m) * inv);
        if (greedy && pt == m) {
            const int32_t k = (int32_t)peek(&mine[i].arg);
            best = k < best ? k : best;
        }
    }
    total = wave_sum(total);
    if (greedy)
        for (int i = kWave / 2; i; i >>= 1) {
            const int32_t y = __shfl_xor(best, i);
            best = y < best ? y : best;
        }
    int32_t say = kRefuse;
    float logp = 0.0f;
    if (!(total > 0.0) || !(m < INFINITY)) {
        say = kBad;
    } else if (known) {
        const double zx = ((double)z_token - m) * inv, p = exp(zx) / total;
        logp = (float)(zx - log(total));
        if (!greedy && fabs(weight - p) <= kClear * p) {
            double sure = exp(zx) / sum_again(z, a.vocab, m, inv, lane);
            if (fabs(weight - sure) <= kClearer * sure) {
                double all = 0.0;
                for (int32_t i = lane; i < a.vocab; i += kWave)
                    all += exp(((double)to_f32(z[i]) - m) * inv);
                sure = exp(zx) / wave_sum(all);
            }
            say = weight < sure ? kAccept : kRefuse;
        } else {
            say = (greedy ? token == best : weight < p) ? kAccept : kRefuse;
        }
    }
    if (lane == 0) {
        sp.rows[r] = Row{total, m, logp, best, say, {0, 0}};
        if (say != kAccept && t < d)
            __hip_atomic_fetch_min(sp.stop + b, t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// What the rows decided, for one request.
struct Outcome {
    int32_t d, at;    // at: the row that the last token comes from
    int32_t out;      // that row's draft token (-1: none)
    float u;          // the draw's random number
    Row row;          // the row
    bool none, bad;   // nothing to commit; because of a bad input
};

// The same on every wavefront: each reads what it takes. Lane t looks at row
// t (then at row t + 64, ...), all its loads issued at once; what rows past
// the last token hold (some other call's verdicts) is not used.
__device__ __forceinline__ Outcome outcome_of(const VerifyArgs &a, const Space &sp, int32_t b)
{
    Outcome o;
    const int64_t r = (int64_t)b * a.rows;
    const int lane = threadIdx.x % kWave;
    o.d = a.draft_len[b];
    o.u = a.uniform[r + a.rows - 1];
    const float tf = temperature(a, b);
    const bool greedy = tf == 0.0f;
    bool bad = !(greedy || (tf >= FLT_MIN && tf <= FLT_MAX)) || o.d < -1 || o.d >= a.rows;
    o.at = o.d;
    o.out = -1;
    o.row = Row{};
    bool found = false;
    for (int32_t base = 0; base < a.rows; base += kWave) {
        const int32_t t = base + lane, in = t < a.rows ? t : a.rows - 1;
        const Row row = sp.rows[r + in];
        const float u = a.uniform[r + in];
        const int32_t x = in < a.rows - 1 ? a.draft[(int64_t)b * (a.rows - 1) + in] : -1;
        if (t < o.d && (x < 0 || x >= a.vocab || (!greedy && !(u >= 0.0f && u < 1.0f))))
            bad = true;
        const uint64_t ends = __ballot(t == o.d || (t < o.d && row.verdict != kAccept));
        if (ends && !found) {
            found = true;
            const int k = __builtin_ctzll(ends);
            o.at = base + k;
            o.out = o.at < o.d ? __shfl(x, k) : -1;
            o.row.total = __shfl(row.total, k);
            o.row.top = __shfl(row.top, k);
            o.row.arg = __shfl(row.arg, k);
            o.row.verdict = __shfl(row.verdict, k);
        }
    }
    if (!greedy && o.d >= 0 && !(o.u >= 0.0f && o.u < 1.0f))
        bad = true;
    o.bad = __any(bad) || (o.d >= 0 && o.row.verdict == kBad);
    o.none = o.bad || o.d < 0;
    return o;
}

// Writes a request's outputs but for the last token, and clears its counters;
// `threads` threads, this one the `first`.
__device__ __forceinline__ void finish(const VerifyArgs &a, const Space &sp, int32_t b,
                                       const Outcome &o, int32_t first, int32_t threads)
{
    const int64_t r = (int64_t)b * a.rows;
    for (int32_t t = first; t < a.rows; t += threads) {
        sp.arrived[r + t] = 0;
        if (!o.none && t == o.at)
            continue;
        const bool drafted = !o.none && t < o.at;
        a.out_tokens[r + t] = drafted ? a.draft[(int64_t)b * (a.rows - 1) + t] : -1;
        if (a.out_logprobs)
            a.out_logprobs[r + t] = drafted ? sp.rows[r + t].logp : 0.0f;
    }
    if (first == 0) {
        a.out_accepted[b] = o.none ? 0 : o.at;
        a.out_counts[b] = o.none ? 0 : o.at + 1;
        sp.stop[b] = kNever;
        sp.drawn[b] = 0;
        if (o.bad)
            atomicOr(a.err, (uint32_t)kErrBlock);
    }
}

// The last token; one thread.
__device__ __forceinline__ void commit(const VerifyArgs &a, int32_t b, const Outcome &o,
                                       int32_t token, double logp)
{
    a.out_tokens[(int64_t)b * a.rows + o.at] = token;
    if (a.out_logprobs)
        a.out_logprobs[(int64_t)b * a.rows + o.at] = (float)logp;
}

// Weight of token i, logit z, of the row a request draws from: `out` is left
// out, and with q only what exceeds it (scaled by the row's total) counts.
__device__ __forceinline__ double weight_of(float z, int32_t i, double top, double inv,
                                            int32_t out, const float *q, double total)
{
    const double w = i == out ? 0.0 : exp(((double)z - top) * inv);
    if (!q)
        return w;
    const double e = w - (double)q[i] * total;
    return e > 0.0 ? e : 0.0;
}

// One wavefront per unit of 64 E logits of the row that a request draws from,
// kWaves units a workgroup. EXCESS 0: sums of the weights; the last workgroup
// of a request without q at that row draws. EXCESS 1 (a second launch, when
// there are drafter probabilities): sums of the excess over q, whose total of
// the weights the first launch left. Measured: 32 us for 64 rows of 151,936
// logits (12 of them the 64-bit exponentials, 9.7 million), 12 us for one of
// 32,000.
template <typename T, int EXCESS, int E>
__global__ __launch_bounds__(kThreads) void draw_kernel(VerifyArgs a, Space sp, int32_t groups)
{
    constexpr int N = 16 / sizeof(T), kUnit = E * kWave, kPer = kUnit / kThreads;
    __shared__ double lds_d[kWaves];
    __shared__ int32_t lds_final, lds_over, lds_piece, lds_pick, lds_last;
    __shared__ double lds_before, lds_goal;
    const int32_t b = blockIdx.x / (uint32_t)groups, group = blockIdx.x % (uint32_t)groups;
    const int32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int32_t draws = (int32_t)pieces_of(a.vocab, kUnit);
    if (EXCESS) {
        // requests that the first launch finished have cleared their row
        // counters; those left have row 0's
        if (sp.arrived[(int64_t)b * a.rows] == 0)
            return;
    }
    const Outcome o = outcome_of(a, sp, b);
    const float tf = temperature(a, b);
    if (o.none || tf == 0.0f) {
        if (group == 0) {
            finish(a, sp, b, o, tid, kThreads);
            if (!o.none && tid == 0)
                commit(a, b, o, o.row.arg, -log(o.row.total));
        }
        return;
    }
    const T *z = (const T *)a.logits + ((int64_t)b * a.rows + o.at) * a.stride;
    const double inv = 1.0 / (double)tf, top = o.row.top;
    const float *q = claim_of(a, b, o.at, o.d);
    const int32_t out = q ? -1 : o.out;
    double total = 0.0;
    if (EXCESS) {
        double part = 0.0;
        for (int32_t i = tid; i < draws; i += kThreads)
            part += sp.weights[(int64_t)b * draws + i];
        total = block_sum(part, lds_d);
    }
    const float *over = EXCESS ? q : nullptr;
    double *sums = (EXCESS ? sp.excess : sp.weights) + (int64_t)b * draws;
    const int32_t unit = group * kWaves + wave;
    if (unit < draws) {
        double part = 0.0;
        const int32_t lo = unit * kUnit + lane * N;
        float x[E];
#pragma unroll
        for (int w = 0; w < E / N; ++w) {
            const int32_t i = lo + w * (kWave * N);
            if (i <= a.vocab - N) {
                const Word<T> y = *(const Word<T> *)(z + i);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    x[w * N + k] = to_f32(y.x[k]);
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k)
                    x[w * N + k] = i + k < a.vocab ? to_f32(z[i + k]) : 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int32_t i = lo + k / N * (kWave * N) + k % N;
            if (i < a.vocab)
                part += weight_of(x[k], i, top, inv, out, over, total);
        }
        part = wave_sum(part);
        if (lane == 0) {
            poke(sums + unit, part);
            asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
        }
    }
    __syncthreads();  // every wavefront's sum is stored
    if (!EXCESS && q)
        return;
    if (tid == 0)
        lds_final = arrive(sp.drawn + b) == groups - 1;
    __syncthreads();
    // (nothing below writes this word: other wavefronts may read it late)
    if (!lds_final)
        return;

    // the last workgroup: one wavefront finds the unit that holds the goal,
    // the others write what is known already
    if (tid >= kWave)
        finish(a, sp, b, o, tid - kWave, kThreads - kWave);
    else {
        // a lane takes `per` units in a row: first whose share holds the goal,
        // then which of its units
        const int32_t per = (draws + kWave - 1) / kWave;
        const auto share = [&] {
            double s = 0.0;
#pragma unroll 8
            for (int32_t i = tid * per; i < (tid + 1) * per; ++i)
                s += i < draws ? peek(sums + i) : 0.0;
            return s;
        };
        double s = share(), all = wave_sum(s);
        if (EXCESS && !(all > 0.0)) {  // (then it is 0)
            // nothing exceeds q: draw from the weights
            over = nullptr;
            sums = sp.weights + (int64_t)b * draws;
            s = share();
            all = wave_sum(s);
        }
        const double goal = (double)o.u * all;
        double before = 0.0;
        int32_t at = -1;
        // the first of 64 shares whose running sum passes the goal (the last
        // with a weight where rounding left none); `before`: what precedes it
        const auto find = [&](double v) {
            double run = v;  // inclusive
            for (int i = 1; i < kWave; i <<= 1) {
                const double y = __shfl_up(run, i);
                if (tid >= i)
                    run += y;
            }
            const uint64_t past = __ballot(v > 0.0 && before + run > goal);
            const uint64_t live = __ballot(v > 0.0);
            if (!live)
                return -1;
            const int k = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(live);
            before += __shfl(run, k) - __shfl(v, k);
            return k;
        };
        int32_t from = 0, count = draws;
        int k = find(s);
        if (k >= 0) {
            from = k * per;
            count = from + per < draws ? per : draws - from;
            // (more than 64 units a lane: the same again with shares of them)
            while (count > kWave) {
                const int32_t step = (count + kWave - 1) / kWave;
                double v = 0.0;
                for (int32_t i = tid * step; i < (tid + 1) * step && i < count; ++i)
                    v += peek(sums + from + i);
                k = find(v);
                count = k * step + step < count ? step : count - k * step;
                from += k * step;
            }
            k = find(tid < count ? peek(sums + from + tid) : 0.0);
            at = from + k;
        }
        const double at_before = before;
        if (tid == 0) {
            lds_piece = at;
            lds_before = at_before;
            lds_goal = goal;
            lds_pick = 0x7fffffff;
            lds_last = -1;
            lds_over = over != nullptr;
        }
    }
    __syncthreads();
    over = lds_over ? q : nullptr;
    const int32_t from = lds_piece * kUnit + tid * kPer;
    double w[kPer], run = 0.0;
    float y[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const bool in = lds_piece >= 0 && from + k < a.vocab;
        y[k] = in ? to_f32(z[from + k]) : 0.0f;
        w[k] = in ? weight_of(y[k], from + k, top, inv, out, over, total) : 0.0;
        run += w[k];
    }
    // exclusive running sum over the threads
    double incl = run;
    for (int i = 1; i < kWave; i <<= 1) {
        const double x = __shfl_up(incl, i);
        if (lane >= i)
            incl += x;
    }
    if (lane == kWave - 1)
        lds_d[wave] = incl;
    __syncthreads();
    double before = lds_before + incl - run;
    for (int i = 0; i < wave; ++i)
        before += lds_d[i];
    int32_t pick = 0x7fffffff, last = -1;
    float z_pick = 0.0f, z_last = 0.0f;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (w[k] > 0.0) {
            before += w[k];
            last = from + k;
            z_last = y[k];
            if (before > lds_goal && pick == 0x7fffffff) {
                pick = from + k;
                z_pick = y[k];
            }
        }
    if (pick != 0x7fffffff)
        atomicMin(&lds_pick, pick);
    if (last >= 0)
        atomicMax(&lds_last, last);
    __syncthreads();
    // the thread that holds the token commits it; without any weight at all
    // the token left out had it all
    const int32_t token = lds_pick != 0x7fffffff ? lds_pick : lds_last;
    if (token < 0 ? tid == 0 : (pick == token || (lds_pick == 0x7fffffff && last == token))) {
        const int32_t x = token < 0 ? (out >= 0 ? out : 0) : token;
        const float zx = token < 0 ? to_f32(z[x]) : (pick == token ? z_pick : z_last);
        commit(a, b, o, x, ((double)zx - top) * inv - log(o.row.total));
    }
}

template <typename K>
hipError_t start(K kernel, int threads, const VerifyArgs &a, const Space &sp, int64_t groups,
                 int64_t pieces, hipStream_t s)
{
    if (!fits_grid(groups * pieces, threads))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(groups * pieces)), dim3(threads), 0, s, a, sp,
                       pieces);
    return hipGetLastError();
}

template <typename T, int E>
hipError_t launch_draw(const VerifyArgs &a, const Space &sp, hipStream_t s)
{
    const int64_t groups = pieces_of(a.vocab, E * kThreads);
    const hipError_t e =
        start(draw_kernel<T, 0, E>, kThreads, a, sp, a.batch, groups, s);
    if (e != hipSuccess || a.head == 0)
        return e;
    return start(draw_kernel<T, 1, E>, kThreads, a, sp, a.batch, groups, s);
}

template <typename T>
hipError_t launch_typed(const VerifyArgs &a, hipStream_t s)
{
    const Space sp = space_of((char *)a.stats, a.max_batch, a.max_rows, a.vocab, nullptr);
    // 8,192 logits a piece from kManyPieces of them on, else 2,048. A few pieces
    // leave the chip empty, and the short ones are read sooner (the call, one row
    // of 32,000: 16.8 us short, 17.4 long). Many short ones cost more to count in
    // and to join than they spread: 20 long pieces 18.2 us both ways, 76 of them
    // 21.5 short and 19.2 long, 304 29.8 and 21.6, 4,864 57.8 and 43.7. A row that
    // one short piece holds takes it at any number (64 x 16 rows of 1,500: 18.4
    // and 19.5).
    constexpr int kWide = 8192 / (16 / sizeof(T)) / kThreads;
    const int64_t rows = (int64_t)a.batch * a.rows, wide = pieces_of(a.vocab, 8192);
    hipError_t e = wide * rows >= kManyPieces && a.vocab > kMinPiece
                       ? start(stats_kernel<T, kWide>, kThreads, a, sp, rows, wide, s)
                       : start(stats_kernel<T, kWide / 4>, kThreads, a, sp, rows,
                               pieces_of(a.vocab, kMinPiece), s);
    // units of 2,048 logits to draw from, or of 512 while they are few and a
    // unit's exponentials are what is waited for (the call, two rows a request:
    // 0.15 million logits 19.5 us with 512, 24.7 with 2,048; 1.2 million 37.5 and
    // 37.9; 1.6 million 31.7 and 31.2; 2.4 million 35.1 and 30.2; 9.7 million 72.5
    // and 45.0)
    if (e == hipSuccess)
        e = (int64_t)a.batch * a.vocab >= (2 << 20) ? launch_draw<T, 32>(a, sp, s)
                                                     : launch_draw<T, 8>(a, sp, s);
    return e;
}

}  // namespace

size_t verify_workspace(int32_t batch, int32_t rows, int32_t vocab)
{
    size_t size;
    (void)space_of(nullptr, batch, rows, vocab, &size);
    return size;
}

hipError_t verify_clear(void *ws, int32_t batch, int32_t rows, int32_t vocab, hipStream_t s)
{
    const Space sp = space_of((char *)ws, batch, rows, vocab, nullptr);
    hipError_t e = hipMemsetAsync(sp.arrived, 0, (char *)sp.stop - (char *)sp.arrived, s);
    if (e == hipSuccess)
        e = hipMemsetAsync(sp.stop, kNever & 0xff, batch * sizeof(int32_t), s);
    return e;
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
