// Verification of a tree of drafted tokens against the target model's logits,
// for gfx950 (MI355X).
//
// Mathematics. The walk starts at the root; at node v with the softmax p of
// its logits row, its children come in index order: child c, token x, is
// accepted when u_c R < p(x), R being what the children refused before it have
// left of 1 (a token refused already has nothing left), and the walk goes on
// there. Where no child is accepted a token is drawn from p without the refused
// ones. This is the chain's rule with more than one try, and commits the
// target's distribution: a child that is come to, with probability R, is taken
// in p(x) / R of the cases.
//
// Of the rows only those on the path are needed, and which they are comes out
// row by row. Two ways to read them:
//  - all rows at once (rows_kernel), a piece of a row a workgroup; the
//    workgroup that completes a row decides which child it leads to, and the
//    path is a walk over these decisions. One round trip, however deep;
//  - the path alone (walk_kernel), a row after the other by a team of workgroups a
//    request: nothing is read that is not needed.
// The row that the walk ends at is then read once more, in 64 bits, for the
// draw (draw_kernel), as in pld_verify.hip.
//
// Decisions are made in 64 bits from a 32-bit sum Z of the weights, whose
// relative error is below 48 * 2^-23 (pld_verify.hip derives it). R carries the
// error of Z as it is, so a decision within 2^-17 u Z of its edge is made again
// from a sum with 64-bit arguments, and within 2^-22 from one with 64-bit
// exponentials.

#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "pld_tree_walk.h"
#include "pld_verify_device.h"

namespace pld {

namespace {

// A node's row, decided; in the place of a Row.
struct Node {
    double total;    // sum of the weights exp((z - top) / T)
    float top;
    int32_t arg;     // greedy: the lowest index of the largest logit
    int32_t next;    // the child accepted, 0: none, -1: a row that holds no distribution
    int32_t pad[3];
};
static_assert(sizeof(Node) == sizeof(Row), "");

constexpr int kParts = WaveTree::kParts;

// What a request's blocks say, checked: rows of the tree (0: none), -1 bad.
__device__ __forceinline__ int32_t nodes_of(const VerifyArgs &a, int32_t b)
{
    const int32_t d = a.draft_len[b];
    return d < -1 || d >= a.rows ? -1 : d + 1;
}

// The drafted nodes as a wavefront holds them: node 64 i + l on lane l.
struct Draft {
    int32_t up[kParts];     // parent, -1 for the root and for what is no node
    int32_t token[kParts];
    float u[kParts];

    // true where something in it is bad
    __device__ __forceinline__ bool load(const TreeVerifyArgs &a, int32_t b, int32_t n, bool greedy,
                                         int lane)
    {
        const int64_t r = (int64_t)b * (a.v.rows - 1) - 1;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int32_t t = i * kWave + lane;
            up[i] = -1;
            token[i] = 0;
            u[i] = 0.0f;
            if (t > 0 && t < n) {
                const int32_t p = a.parent ? a.parent[r + t] : t - 1;
                token[i] = a.v.draft[r + t];
                u[i] = a.v.uniform[(int64_t)b * a.v.rows + t - 1];
                const bool fine = p >= 0 && p < t && token[i] >= 0 && token[i] < a.v.vocab &&
                                  (greedy || (u[i] >= 0.0f && u[i] < 1.0f));
                bad |= !fine;
                up[i] = fine ? p : -1;
                token[i] = fine ? token[i] : 0;
            }
        }
        return __any(bad);
    }
};

// The value that lane `from` of part `part` holds; both the same on every lane.
template <typename X>
__device__ __forceinline__ X pick(const X (&x)[kParts], int32_t t)
{
    X y = x[0];
#pragma unroll
    for (int i = 1; i < kParts; ++i)
        y = t / kWave == i ? x[i] : y;
    return __shfl(y, t % kWave);
}

// The child of node v that its row leads to, or 0; one wavefront, the same on
// every lane. z: the row; zx: the logits of the children's tokens; m, total,
// best: the row's largest logit, the sum of its weights (32-bit), its argmax.
template <typename T>
__device__ __forceinline__ int32_t child_of(const Draft &d, const T *z, int32_t vocab, int32_t v,
                                            const float (&zx)[kParts], float m, double total,
                                            double inv, bool greedy, int32_t best, int lane)
{
    if (greedy) {
        int32_t on = 0;
#pragma unroll
        for (int i = kParts - 1; i >= 0; --i) {
            const uint64_t hit = __ballot(d.up[i] == v && d.token[i] == best);
            if (hit)
                on = i * kWave + __builtin_ctzll(hit);
        }
        return on;
    }
    double w[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i)
        w[i] = d.up[i] == v ? exp(((double)zx[i] - m) * inv) : 0.0;
    for (int sure = 0;; ++sure) {
        const double slack = sure == 0 ? kClear : (sure == 1 ? kClearer : 0.0);
        double left = total;
        bool close = false;
        double now[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            now[i] = w[i];
        int32_t on = 0;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            uint64_t kids = __ballot(d.up[i] == v);
            while (kids && !on && !close) {
                const int k = __builtin_ctzll(kids);
                kids &= kids - 1;
                const double wk = __shfl(now[i], k);
                const double uk = (double)__shfl(d.u[i], k);
                const int32_t x = __shfl(d.token[i], k);
                if (!(wk > 0.0))
                    continue;
                if (slack > 0.0 && fabs(uk * left - wk) <= slack * uk * total)
                    close = true;
                else if (uk * left < wk)
                    on = i * kWave + k;
                left -= wk;
                // (the same token once more has nothing left)
#pragma unroll
                for (int j = 0; j < kParts; ++j)
                    now[j] = d.token[j] == x ? 0.0 : now[j];
            }
        }
        if (!close)
            return on;
        if (sure == 0) {
            total = sum_again(z, vocab, m, inv, lane);
        } else {
            double all = 0.0;
            for (int32_t i = lane; i < vocab; i += kWave)
                all += exp(((double)to_f32(z[i]) - m) * inv);
            total = wave_sum(all);
        }
    }
}

// The logits of node v's children's tokens.
template <typename T>
__device__ __forceinline__ void child_logits(const Draft &d, const T *z, int32_t v,
                                             float (&zx)[kParts])
{
#pragma unroll
    for (int i = 0; i < kParts; ++i)
        zx[i] = d.up[i] == v ? to_f32(z[d.token[i]]) : 0.0f;
}

// What a workgroup finds in a piece of a row: on thread 0.
struct Found {
    float top, sum;
    int32_t arg;
};
struct Scratch {
    float top[kWaves], sum[kWaves];
    int32_t arg[kWaves];
};

// The largest logit of a piece, where it is (greedy) and the sum of the
// weights, W 16-byte words a thread, in one read. Every wavefront but the first
// may go on when it returns; s is free again after the next barrier.
template <typename T, int W>
__device__ __forceinline__ Found search(const T *z, int32_t vocab, int32_t piece, float c,
                                        bool greedy, Scratch &s)
{
    constexpr int N = 16 / sizeof(T);
    const int32_t tid = threadIdx.x;
    const int wave = tid / kWave, lane = tid % kWave;
    float x[W * N];
    float top = -INFINITY;
    const int32_t lo = piece * (W * N * kThreads) + tid * N;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int32_t i = lo + w * (kThreads * N);
        if (i <= vocab - N) {
            const Word<T> y = *(const Word<T> *)(z + i);
#pragma unroll
            for (int k = 0; k < N; ++k)
                x[w * N + k] = to_f32(y.x[k]);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
                x[w * N + k] = i + k < vocab ? to_f32(z[i + k]) : -INFINITY;
        }
    }
#pragma unroll
    for (int k = 0; k < W * N; ++k)
        top = fmaxf(top, x[k]);
    top = wave_max(top);
    if (lane == 0)
        s.top[wave] = top;
    __syncthreads();
    top = s.top[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        top = fmaxf(top, s.top[w]);
    // (as in pld_verify.hip: one operation a logit, what rounding takes off the
    // common exponent put back into the sum, or two where logits are far)
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
        s.sum[wave] = sum;
        s.arg[wave] = arg;
    }
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            sum += s.sum[w];
            arg = s.arg[w] < arg ? s.arg[w] : arg;
        }
        sum *= __builtin_amdgcn_exp2f(-rest);
    }
    return Found{top, sum, arg};
}

// A piece's findings, for the workgroup that joins the row; one thread. Its
// stores are complete when it counts itself in.
__device__ __forceinline__ void leave(Piece *at, const Found &f, bool greedy)
{
    poke(&at->top_sum, (unsigned long long)__float_as_uint(f.top) << 32 | __float_as_uint(f.sum));
    if (greedy)
        poke(&at->arg, (unsigned long long)(uint32_t)f.arg);
}

// Joins the pieces of node t's row and decides which child it leads to; one
// wavefront, the same on every lane.
template <typename T>
__device__ __forceinline__ int32_t decide(const VerifyArgs &a, const Space &sp, const Draft &d,
                                          int32_t b, int32_t t, const T *z,
                                          const float (&zx)[kParts], uint32_t pieces, float tf,
                                          int lane)
{
    const bool greedy = tf == 0.0f;
    const double inv = greedy ? 1.0 : 1.0 / (double)tf;
    const int64_t r = (int64_t)b * a.rows + t;
    const Piece *const mine = sp.pieces + r * pieces;
    float m = -INFINITY;
    for (uint32_t i = lane; i < pieces; i += kWave)
        m = fmaxf(m, __uint_as_float((uint32_t)(peek(&mine[i].top_sum) >> 32)));
    m = wave_max(m);
    int32_t best = 0x7fffffff;
    double total = 0.0;
    for (uint32_t i = lane; i < pieces; i += kWave) {
        const unsigned long long y = peek(&mine[i].top_sum);
        const float pt = __uint_as_float((uint32_t)(y >> 32));
        const float ps = __uint_as_float((uint32_t)y);
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
    int32_t next = -1;
    if (total > 0.0 && m < INFINITY)
        next = child_of(d, z, a.vocab, t, zx, m, total, inv, greedy, best, lane);
    if (lane == 0)
        ((Node *)sp.rows)[r] = Node{total, m, best, next, {0, 0, 0}};
    return next;
}

// All rows at once: one workgroup per piece of a row. 16 trees of 32 rows of
// 50,257 f16 logits: 21.7 us, 51 MB at 2.4 TB/s; 16 rows of 32,000 f32 logits: 7.1.
template <typename T, int W>
__global__ __launch_bounds__(kThreads) void rows_kernel(TreeVerifyArgs ta, Space sp,
                                                        uint32_t pieces)
{
    const VerifyArgs &a = ta.v;
    __shared__ Scratch lds;
    const int32_t piece = blockIdx.x % pieces, lane = threadIdx.x % kWave;
    const uint32_t order = blockIdx.x / pieces;
    const int32_t b = order % (uint32_t)a.batch, t = order / (uint32_t)a.batch;
    const int32_t n = nodes_of(a, b);
    if (t >= n)
        return;
    const int64_t r = (int64_t)b * a.rows + t;
    const T *z = (const T *)a.logits + r * a.stride;
    const float tf = temperature(a, b);
    const bool greedy = tf == 0.0f;
    const Found f =
        search<T, W>(z, a.vocab, piece, kLog2e / (greedy ? 1.0f : tf), greedy, lds);
    if (threadIdx.x >= kWave)
        return;  // one wavefront counts the piece in, and decides if it is the last
    int32_t count = 0;
    if (lane == 0) {
        leave(sp.pieces + r * pieces + piece, f, greedy);
        count = arrive(sp.arrived + r);
    }
    if (__builtin_amdgcn_readfirstlane(count) != (int32_t)pieces - 1)
        return;
    Draft d;
    (void)d.load(ta, b, n, greedy, lane);
    float zx[kParts];
    child_logits(d, z, t, zx);
    (void)decide(a, sp, d, b, t, z, zx, pieces, tf, lane);
}

constexpr int32_t kThere = -1;     // `stop` once a walk has ended
constexpr int32_t kDone = 1 << 16;  // `arrived` counts pieces taken below, pieces done above

// The path alone: a team of workgroups a request. They take the pieces of the
// walk's row one by one; who completes the row decides where the walk goes on,
// and says so in `stop`. A workgroup that finds every piece of the row taken
// waits for that. It waits for workgroups that run and wait for nothing
// themselves while they have a piece: the walk ends however many of a team the
// chip has room for, one included. 64 trees of up to 64 rows of 151,936 bf16 logits:
// 58 us, 47 MB read, 6 to 7 us a row of the longest path: taking a piece, reading,
// counting in, joining and being seen are a round trip each. (One workgroup of 1,024
// threads a request: 97, its exponentials bound it.)
template <typename T, int W>
__global__ __launch_bounds__(kThreads) void walk_kernel(TreeVerifyArgs ta, Space sp,
                                                        uint32_t pieces, uint32_t team)
{
    const VerifyArgs &a = ta.v;
    __shared__ Scratch lds;
    __shared__ int32_t lds_piece, lds_node;
    const int32_t b = blockIdx.x / team, tid = threadIdx.x, lane = tid % kWave;
    const bool first = tid < kWave;
    const int32_t n = nodes_of(a, b);
    if (n <= 0)
        return;
    const float tf = temperature(a, b);
    const bool greedy = tf == 0.0f;
    const float c = kLog2e / (greedy ? 1.0f : tf);
    Draft d;
    if (d.load(ta, b, n, greedy, lane))
        return;  // (the draw finds the same)
    int32_t *const stop = sp.stop + b;
    int32_t node = 0;
    for (;;) {
        const int64_t r = (int64_t)b * a.rows + node;
        if (tid == 0)
            lds_piece = __hip_atomic_fetch_add(sp.arrived + r, 1, __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT) & (kDone - 1);
        __syncthreads();
        const int32_t piece = lds_piece;
        if (piece >= (int32_t)pieces) {
            if (tid == 0) {
                int32_t to = peek(stop);
                while (to == (node ? node : kNever)) {
                    __builtin_amdgcn_s_sleep(2);
                    to = peek(stop);
                }
                lds_node = to;
            }
            __syncthreads();
            node = lds_node;
            if (node == kThere)
                return;
            continue;
        }
        const T *z = (const T *)a.logits + r * a.stride;
        float zx[kParts];
        if (first)
            child_logits(d, z, node, zx);
        const Found f = search<T, W>(z, a.vocab, piece, c, greedy, lds);
        if (first) {
            int32_t count = 0, next = node;
            if (lane == 0) {
                leave(sp.pieces + r * pieces + piece, f, greedy);
                asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
                count = __hip_atomic_fetch_add(sp.arrived + r, kDone, __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT) / kDone;
            }
            if (__builtin_amdgcn_readfirstlane(count) == (int32_t)pieces - 1) {
                next = decide(a, sp, d, b, node, z, zx, pieces, tf, lane);
                next = next > 0 ? next : kThere;
                if (lane == 0)
                    poke(stop, next);
            }
            if (lane == 0)
                lds_node = next;
        }
        __syncthreads();
        node = lds_node;
        if (node == kThere)
            return;
    }
}

// What the rows decided, for one request; the same on every lane.
struct Path {
    int32_t n;           // nodes, -1 bad
    int32_t at, steps;   // the node that the token is drawn at, and its depth
    bool none, bad;      // nothing to commit; because of a bad input
};

// Every wavefront reads what it takes. `to`: where the path's nodes go, or
// null.
__device__ __forceinline__ Path path_of(const TreeVerifyArgs &ta, const Space &sp, int32_t b,
                                        Draft &d, int lane, uint16_t *to)
{
    const VerifyArgs &a = ta.v;
    Path p;
    p.n = nodes_of(a, b);
    p.at = p.steps = 0;
    const float tf = temperature(a, b), u = a.uniform[(int64_t)b * a.rows + a.rows - 1];
    const bool greedy = tf == 0.0f;
    const Node *node = (const Node *)sp.rows + (int64_t)b * a.rows;
    int32_t next[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int32_t t = i * kWave + lane;
        next[i] = t < p.n ? node[t].next : 0;
    }
    p.bad = d.load(ta, b, p.n, greedy, lane) || p.n < 0 ||
            !(greedy || (tf >= FLT_MIN && tf <= FLT_MAX)) ||
            (!greedy && p.n > 0 && !(u >= 0.0f && u < 1.0f));
    if (!p.bad && p.n > 0) {
        for (;;) {
            if (to)
                to[p.steps] = (uint16_t)p.at;
            const int32_t x = pick(next, p.at);
            p.bad = x < 0;
            if (x <= p.at || x >= p.n)
                break;
            p.at = x;
            ++p.steps;
        }
    }
    p.none = p.bad || p.n <= 0;
    return p;
}

// Log probability of token x at a decided row.
template <typename T>
__device__ __forceinline__ float log_of(const VerifyArgs &a, const Space &sp, int32_t b,
                                        int32_t node, int32_t x, double inv)
{
    const int64_t r = (int64_t)b * a.rows + node;
    const Node row = ((const Node *)sp.rows)[r];
    const double z = to_f32(((const T *)a.logits)[r * a.stride + x]);
    return (float)((z - row.top) * inv - log(row.total));
}

// Writes a request's outputs but for the last token, and clears its counters;
// `threads` threads, this one the `first`. `path`: its nodes.
template <typename T>
__device__ __forceinline__ void finish(const TreeVerifyArgs &ta, const Space &sp, int32_t b,
                                       const Path &p, const uint16_t *path, double inv,
                                       int32_t first, int32_t threads)
{
    const VerifyArgs &a = ta.v;
    const int64_t r = (int64_t)b * a.rows;
    for (int32_t i = first; i < a.rows; i += threads) {
        sp.arrived[r + i] = 0;
        ta.out_path[r + i] = !p.none && i <= p.steps ? path[i] : -1;
        if (!p.none && i == p.steps)
            continue;
        const bool drafted = !p.none && i < p.steps;
        const int32_t x =
            drafted ? a.draft[(int64_t)b * (a.rows - 1) + path[i + 1] - 1] : -1;
        a.out_tokens[r + i] = x;
        if (a.out_logprobs)
            a.out_logprobs[r + i] = drafted ? log_of<T>(a, sp, b, path[i], x, inv) : 0.0f;
    }
    if (first == 0) {
        a.out_accepted[b] = p.none ? 0 : p.steps;
        a.out_counts[b] = p.none ? 0 : p.steps + 1;
        sp.stop[b] = kNever;
        sp.drawn[b] = 0;
        if (p.bad)
            atomicOr(a.err, (uint32_t)kErrBlock);
    }
}

// The last token; one thread.
template <typename T>
__device__ __forceinline__ void commit(const VerifyArgs &a, const Space &sp, int32_t b,
                                       const Path &p, int32_t token, double inv)
{
    a.out_tokens[(int64_t)b * a.rows + p.steps] = token;
    if (a.out_logprobs)
        a.out_logprobs[(int64_t)b * a.rows + p.steps] = log_of<T>(a, sp, b, p.at, token, inv);
}

// One wavefront per unit of 64 E logits of the row that a request draws from,
// kWaves units a workgroup: sums of the weights, without the refused children's;
// the last workgroup of a request draws. 31 us for 64 rows of 151,936 logits, 12 for
// one of 32,000, as in pld_verify.hip; 4.6 where all requests are greedy.
template <typename T, int E>
__global__ __launch_bounds__(kThreads) void draw_kernel(TreeVerifyArgs ta, Space sp,
                                                        int32_t groups)
{
    const VerifyArgs &a = ta.v;
    constexpr int N = 16 / sizeof(T), kUnit = E * kWave, kPer = kUnit / kThreads;
    __shared__ uint16_t lds_path[kTreeRows];
    __shared__ double lds_d[kWaves];
    __shared__ int32_t lds_final, lds_unit, lds_pick, lds_last;
    __shared__ double lds_before, lds_goal;
    const int32_t b = blockIdx.x / (uint32_t)groups, group = blockIdx.x % (uint32_t)groups;
    const int32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int32_t draws = (int32_t)pieces_of(a.vocab, kUnit);
    Draft d;
    const Path p = path_of(ta, sp, b, d, lane, wave == 0 ? lds_path : nullptr);
    const float tf = temperature(a, b);
    const double inv = tf == 0.0f ? 1.0 : 1.0 / (double)tf;
    if (p.none || tf == 0.0f) {
        if (group == 0) {
            __syncthreads();
            finish<T>(ta, sp, b, p, lds_path, inv, tid, kThreads);
            if (!p.none && tid == 0)
                commit<T>(a, sp, b, p, ((const Node *)sp.rows)[(int64_t)b * a.rows + p.at].arg,
                          inv);
        }
        return;
    }
    const int64_t r = (int64_t)b * a.rows + p.at;
    const T *z = (const T *)a.logits + r * a.stride;
    const double top = ((const Node *)sp.rows)[r].top;
    double *sums = sp.weights + (int64_t)b * draws;
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
                    x[w * N + k] = i + k < a.vocab ? to_f32(z[i + k]) : -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const bool mine = d.up[i] == p.at && d.token[i] / kUnit == unit;
            for (uint64_t out = __ballot(mine); out; out &= out - 1) {
                const int32_t y = __shfl(d.token[i], __builtin_ctzll(out));
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (lo + k / N * (kWave * N) + k % N == y)
                        x[k] = -INFINITY;
            }
        }
#pragma unroll
        for (int k = 0; k < E; ++k)
            part += exp(((double)x[k] - top) * inv);
        part = wave_sum(part);
        if (lane == 0) {
            poke(sums + unit, part);
            asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
        }
    }
    __syncthreads();  // every wavefront's sum is stored
    if (tid == 0)
        lds_final = arrive(sp.drawn + b) == groups - 1;
    __syncthreads();
    if (!lds_final)
        return;

    // the last workgroup: one wavefront finds the unit that holds the goal,
    // the others write what is known already
    if (wave > 0) {
        finish<T>(ta, sp, b, p, lds_path, inv, tid - kWave, kThreads - kWave);
    } else {
        // a lane takes `per` units in a row: first whose share holds the goal,
        // then which of its units
        double before = 0.0, goal = 0.0;
        int32_t from = 0, count = draws;
        bool live = true;
        for (bool first = true; live; first = false) {
            const int32_t per = (count + kWave - 1) / kWave;
            double s = 0.0;
#pragma unroll 8
            for (int32_t i = lane * per; i < (lane + 1) * per; ++i)
                s += i < count ? peek(sums + from + i) : 0.0;
            double run = s;  // inclusive
            for (int i = 1; i < kWave; i <<= 1) {
                const double y = __shfl_up(run, i);
                if (lane >= i)
                    run += y;
            }
            if (first)
                goal = (double)a.uniform[(int64_t)b * a.rows + a.rows - 1] *
                       __shfl(run, kWave - 1);
            // the first share whose running sum passes the goal (the last with
            // a weight where rounding left none); `before`: what precedes it
            const uint64_t past = __ballot(s > 0.0 && before + run > goal);
            const uint64_t some = __ballot(s > 0.0);
            live = some != 0;
            const int k = past ? __builtin_ctzll(past) : (live ? 63 - __builtin_clzll(some) : 0);
            before += __shfl(run, k) - __shfl(s, k);
            from += k * per;
            count = per < count - k * per ? per : count - k * per;
            if (per == 1)
                break;
        }
        if (lane == 0) {
            lds_unit = live ? from : -1;
            lds_before = before;
            lds_goal = goal;
            lds_pick = 0x7fffffff;
            lds_last = -1;
        }
    }
    __syncthreads();
    const int32_t from = lds_unit * kUnit + tid * kPer;
    double w[kPer], run = 0.0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const bool in = lds_unit >= 0 && from + k < a.vocab;
        w[k] = in ? exp(((double)to_f32(z[from + k]) - top) * inv) : 0.0;
    }
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const bool mine = d.up[i] == p.at && d.token[i] / kUnit == lds_unit;
        for (uint64_t out = __ballot(mine); out; out &= out - 1) {
            const int32_t y = __shfl(d.token[i], __builtin_ctzll(out));
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (from + k == y)
                    w[k] = 0.0;
        }
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        run += w[k];
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
    int32_t token = 0x7fffffff, last = -1;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (w[k] > 0.0) {
            before += w[k];
            last = from + k;
            if (before > lds_goal && token == 0x7fffffff)
                token = from + k;
        }
    if (token != 0x7fffffff)
        atomicMin(&lds_pick, token);
    if (last >= 0)
        atomicMax(&lds_last, last);
    __syncthreads();
    if (tid != 0)
        return;
    token = lds_pick != 0x7fffffff ? lds_pick : lds_last;
    // without any weight at all the refused tokens had it all: the likeliest
    if (token < 0) {
        float high = -INFINITY;
        for (int32_t t = 1; t < p.n; ++t) {
            const int64_t i = (int64_t)b * (a.rows - 1) + t - 1;
            if ((ta.parent ? ta.parent[i] : t - 1) != p.at)
                continue;
            const float y = to_f32(z[a.draft[i]]);
            if (y > high) {
                high = y;
                token = a.draft[i];
            }
        }
        token = token < 0 ? 0 : token;
    }
    commit<T>(a, sp, b, p, token, inv);
}

template <typename K, typename... X>
hipError_t start(K kernel, int threads, int64_t groups, hipStream_t s, X... x)
{
    if (!fits_grid(groups, threads))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)groups), dim3(threads), 0, s, x...);
    return hipGetLastError();
}

template <typename T, int E>
hipError_t launch_draw(const TreeVerifyArgs &a, const Space &sp, hipStream_t s)
{
    const int64_t groups = pieces_of(a.v.vocab, E * kThreads);
    return start(draw_kernel<T, E>, kThreads, a.v.batch * groups, s, a, sp, (int32_t)groups);
}

// Bytes of logits (of the padded rows) up to which all rows are read. Measured
// with ragged trees, all rows and the path, the call: 1 tree of 64 rows of 151,936
// bf16 logits 22 us (the same call), 4 trees 28 and 42, 8 (155 MB) 50 and 51, 16 (311
// MB) 70 and 71, 24 80 and 61, 64 239 and 87; 64 of 16 rows (311 MB) 77 and 97; 64 of 32
// rows of 50,257 (206 MB) 62 and 64; 16 full ones of those (51 MB, greedy) 27 and 62.
// Bytes alone do not place every shape: the path costs a round trip a level and all
// rows cost their live bytes, so many trees of few rows just past the bound take the
// slower side (97 for 77).
constexpr int64_t kAllBytes = 256 << 20;
constexpr int64_t kResident = 2048;      // workgroups of a walk that the chip holds at once

template <typename T, int W>
hipError_t launch_walk(const TreeVerifyArgs &a, const Space &sp, int64_t pieces, hipStream_t s)
{
    const int64_t room = kResident / a.v.batch;
    const int64_t team = pieces < room ? pieces : (room > 1 ? room : 1);
    return start(walk_kernel<T, W>, kThreads, a.v.batch * team, s, a, sp, (uint32_t)pieces,
                 (uint32_t)team);
}

template <typename T>
hipError_t launch_typed(const TreeVerifyArgs &a, hipStream_t s)
{
    const VerifyArgs &v = a.v;
    const Space sp = space_of((char *)v.stats, v.max_batch, v.max_rows, v.vocab, nullptr);
    constexpr int kWide = 8192 / (16 / sizeof(T)) / kThreads;
    const int64_t rows = (int64_t)v.batch * v.rows, wide = pieces_of(v.vocab, 8192);
    const int64_t small = pieces_of(v.vocab, kMinPiece);
    // (both launches or none: the second leaves the counters for the next call)
    if (!fits_grid(v.batch * pieces_of(v.vocab, 8 * kThreads), kThreads))
        return hipErrorInvalidConfiguration;
    hipError_t e;
    if (rows * v.vocab * (int64_t)sizeof(T) > kAllBytes)
        e = launch_walk<T, kWide>(a, sp, wide, s);
    else if (wide * rows >= kManyPieces && v.vocab > kMinPiece)
        e = start(rows_kernel<T, kWide>, kThreads, rows * wide, s, a, sp, (uint32_t)wide);
    else
        e = start(rows_kernel<T, kWide / 4>, kThreads, rows * small, s, a, sp, (uint32_t)small);
    if (e == hipSuccess)
        e = (int64_t)v.batch * v.vocab >= (2 << 20) ? launch_draw<T, 32>(a, sp, s)
                                                    : launch_draw<T, 8>(a, sp, s);
    return e;
}

}  // namespace

hipError_t launch_verify_tree(const TreeVerifyArgs &a, hipStream_t s)
{
    switch (a.v.dtype) {
    case PLD_F32: return launch_typed<float>(a, s);
    case PLD_F16: return launch_typed<_Float16>(a, s);
    default: return launch_typed<__bf16>(a, s);
    }
}

}  // namespace pld
