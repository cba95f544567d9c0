// Attention of the verify block's rows over the paged cache, for gfx950
// (MI355X).
//
// Mathematics. A workgroup takes one request, one kv head, a tile of query
// rows (row m = block row t, query head g of the group: m = t * G + g) and a
// span of positions, tile by tile of positions, with a running maximum m, sum
// l and output O (one pass over the cache):
//   S^T = K Q^T,  P^T = 2^(c S^T - m + kLift),  O^T += V^T P^T,  l += sum P,
// c = scale * log2 e. Both products are 16x16x32 matrix instructions whose
// left operand is the cache as it lies in memory: a lane holds 16 bytes of a
// K row (positions x dims) or of a V row (dims x positions; that is why V
// pages hold positions side by side), so nothing is transposed. The result
// layout of S^T (lane: one query row, positions 4 (lane / 16) + r) is the right
// operand's layout of P^T once the positions of a tile are dealt to the K rows
// in the matching order, so P never leaves its lane either.
//
// m is raised only when a score passes it by kSlack (the sum and O are then
// rescaled); P is lifted by 2^kLift, so that in fp16 probabilities down to
// 2^-26 of the row's largest keep all their bits and 2^(kLift + kSlack) stays
// below 65504. A probability is rounded to T, half a step, because it is an
// operand of the second product; l sums it unrounded, in 32 bits. (16 requests of
// 131,072 positions and 512 query rows in bf16 are 0.0018 off the 64-bit result so,
// relative to its norm; all in 32 bits and rounded once, 0.0017: the output's own
// rounding.)
//
// TREE: the block is a tree of drafted tokens. Every row sees the history up
// to the root's cell, and of the cells behind it those of its own ancestors
// and its own: a row's branch, a string of bits in LDS, one a cell. Only tiles
// that reach behind the root look at it. It is built by workgroups that come
// to such a tile, in rounds that double the ancestors known (as many as the
// logarithm of the deepest branch). Positions, for windows, go by depth.

#pragma once

#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "pld_tree.h"
#include "pld_target_device.h"

namespace pld {

namespace {

constexpr int kWave = 64;
constexpr int kWaves = 4;             // wavefronts of a workgroup
constexpr float kLift = 12.0f;
constexpr float kSlack = 3.0f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

typedef float F4 __attribute__((ext_vector_type(4)));
typedef uint32_t U4 __attribute__((ext_vector_type(4)));
typedef uint32_t U2 __attribute__((ext_vector_type(2)));

// 8 values of T as a matrix operand.
template <typename T> struct Frag;
template <> struct Frag<__bf16> {
    typedef __bf16 V8 __attribute__((ext_vector_type(8)));
    typedef __bf16 V2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ F4 mma(U4 a, U4 b, F4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V8, a),
                                                       __builtin_bit_cast(V8, b), c, 0, 0, 0);
    }
    // bytes 0..1 or 2..3 of w, E4M3, to two values (exact)
    template <bool HI> static __device__ __forceinline__ uint32_t widen(uint32_t w)
    {
        return __builtin_bit_cast(uint32_t,
                                  __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
    }
};
template <> struct Frag<_Float16> {
    typedef _Float16 V8 __attribute__((ext_vector_type(8)));
    typedef _Float16 V2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ F4 mma(U4 a, U4 b, F4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V8, a),
                                                      __builtin_bit_cast(V8, b), c, 0, 0, 0);
    }
    template <bool HI> static __device__ __forceinline__ uint32_t widen(uint32_t w)
    {
        return __builtin_bit_cast(uint32_t,
                                  __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
    }
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    typename Frag<T>::V2 v;
    v[0] = (T)a;
    v[1] = (T)b;
    return __builtin_bit_cast(uint32_t, v);
}

template <typename T>
__device__ __forceinline__ U4 widen8(uint32_t a, uint32_t b)
{
    return U4{Frag<T>::template widen<false>(a), Frag<T>::template widen<true>(a),
              Frag<T>::template widen<false>(b), Frag<T>::template widen<true>(b)};
}

// The factor on the scores. Never 0, where a product of small scales would
// be: 0 times a masked score's -infinity is NaN.
__device__ __forceinline__ float factor(float c)
{
    const float x = fabsf(c);
    return x < FLT_MIN ? FLT_MIN : x;
}

// How a launch splits the positions: spans of `span` positions (a multiple
// of the tile), `splits` of them at most; partial results of a request whose
// positions take more than one.
struct Split {
    int32_t span;
    int32_t least;     // trees: positions that a span of any request has at least
    int32_t splits;
    int32_t m_tiles;   // tiles of query rows
    float *o;          // [batch][kv_heads][splits][m_tiles * 16 MB][D]
    float2 *ml;        // [batch][kv_heads][splits][m_tiles * 16 MB]: m, l
};

// Positions that query rows [m0, m1] of a request see: [lo, hi], and where
// the first span starts.
struct Sight {
    int32_t lo, hi, start;
};

// (A tree's rows stand at the root's position or behind it.)
template <int TK, bool TREE>
__device__ __forceinline__ Sight sight_of(const AttendArgs &a, int32_t length, int32_t t0,
                                          int32_t t1)
{
    Sight s;
    const int32_t first = length - 1 + (TREE ? 0 : t0);
    s.lo = a.window && first >= a.window ? first - a.window + 1 : 0;
    s.hi = length - 1 + t1;
    s.start = s.lo / TK * TK;
    return s;
}

// The branches of a tree's rows, in LDS: a row's string has a word of ones for
// the cells before the root's, then a bit for each node, then a word of zeros;
// behind it its depth.
struct Branches {
    static constexpr int kWords = kTreeRows / 32, kPitch = kWords + 3, kDepth = kWords + 2;
    static constexpr int kLds = kTreeRows * (kPitch * 4 + 2);
    static_assert(kTreeRows == kWaves * kWave, "a thread a node");

    // The branches of nodes 0..n - 1, with the window's part of them (0: all),
    // by the whole workgroup: thread t brings node t's parent (0 for t = 0 and
    // from n on). A barrier stands behind them.
    static __device__ __forceinline__ void build(char *lds, int32_t up, int32_t n, int32_t window)
    {
        uint32_t *const rows = (uint32_t *)lds;
        uint16_t *const ups = (uint16_t *)(rows + kTreeRows * kPitch);
        const int32_t t = threadIdx.x;
        uint32_t *const mine = rows + t * kPitch;
        mine[0] = 0xffffffffu;
        for (int i = 1; i < kDepth; ++i)
            mine[i] = 0;
        mine[1 + t / 32] = 1u << (t & 31);
        ups[t] = (uint16_t)up;
        // a string holds the branch from t up to, not with, `up`
        while (__syncthreads_or(up != 0)) {
            uint32_t w[kWords];
            int32_t next = 0;
            if (up != 0) {
                for (int i = 0; i < kWords; ++i)
                    w[i] = rows[up * kPitch + 1 + i];
                next = ups[up];
            }
            __syncthreads();
            if (up != 0) {
                for (int i = 0; i < kWords; ++i)
                    mine[1 + i] |= w[i];
                ups[t] = (uint16_t)next;
                up = next;
            }
        }
        if (t < n) {
            mine[1] |= 1u;
            int32_t nodes = 0;
            for (int i = 1; i <= kWords; ++i)
                nodes += __popc(mine[i]);
            mine[kDepth] = nodes - 1;
            // a branch's nodes have rising indexes: the window's are the last
            int32_t keep = window ? window : kTreeRows;
            for (int i = kWords; i > 0; --i) {
                uint32_t x = mine[i];
                const int32_t here = __popc(x);
                for (int32_t drop = here - keep; drop > 0; --drop)
                    x &= x - 1;
                mine[i] = x;
                keep -= here < keep ? here : keep;
            }
        }
        __syncthreads();
    }

    // Which of the 32 cells from `cell` on row t's branch holds, `root` being
    // the root's cell; all of those before it.
    static __device__ __forceinline__ uint32_t bits(const char *lds, int32_t t, int32_t cell,
                                                    int32_t root)
    {
        const int32_t at = cell - root + 32;
        if (at <= 0)
            return 0xffffffffu;
        if (at >= 32 + kTreeRows)
            return 0;
        const uint32_t *w = (const uint32_t *)lds + t * kPitch + at / 32;
        return (uint32_t)((((uint64_t)w[1] << 32) | w[0]) >> (at & 31));
    }
    static __device__ __forceinline__ int32_t depth(const char *lds, int32_t t)
    {
        return (int32_t)((const uint32_t *)lds)[t * kPitch + kDepth];
    }
};

// Positions of a request's spans. A tree's are dealt out evenly: a batch with
// ragged lengths has all of its workgroups at work, each on a share of its own
// request, where equal spans leave the short requests' idle: 64 requests of
// 8,192 to 65,536 positions, 96 query rows and 8-bit cells 1,155 us with equal
// spans, 863 so.
template <bool TREE, int GRAIN>
__device__ __forceinline__ int32_t span_of(const Split &sp, const Sight &s)
{
    if (!TREE)
        return sp.span;
    const int32_t even =
        (int32_t)(((int64_t)s.hi - s.start) / sp.splits / GRAIN + 1) * GRAIN;
    return even < sp.least ? sp.least : (even > sp.span ? sp.span : even);
}

// What both kernels share: MB blocks of 16 query rows a wavefront.
template <typename T, typename C, int D, int MB, bool TREE>
struct Tiles {
    static constexpr bool kTree = TREE;
    static constexpr bool kByte = sizeof(C) == 1;
    static constexpr int TK = kByte ? 64 : 32;  // positions of a tile
    static constexpr int kGrain = kWaves * TK;  // a span is a multiple of so many positions
    static constexpr int64_t kSpanBytes = 4 << 20;
    static constexpr int NB = TK / 32;          // 32-position steps of V^T P^T
    static constexpr int CH = 8 * NB;           // positions of a lane's V word
    static constexpr int DB = D / 16;           // blocks of 16 dims
    static constexpr int KW = kByte ? (D + 63) / 64 : D / 32;  // 16-byte words of a K row, a lane
    static constexpr int KS = kByte ? 2 * KW : KW;             // 32-dim steps of K Q^T
    static constexpr int kCells = 16 / (int)sizeof(C);         // of a word
    static constexpr int kCellBytes = (int)sizeof(C);

    // A K row's word w starts here for lane group g. With 8-bit cells a word
    // serves two steps; where the dims are no multiple of 64 the last word
    // reaches back over dims the one before it had.
    static __device__ __forceinline__ int word_of(int w, int g)
    {
        if (kByte && (w + 1) * 64 > D)
            return D - 64 + g * 16;
        return w * (4 * kCells) + g * kCells;
    }
    // The first of the 8 dims of step s that lane group g holds, or -1 where
    // they are such a repetition (their q is zero).
    static __device__ __forceinline__ int dim_of(int s, int g)
    {
        if (!kByte)
            return s * 32 + g * 8;
        const int d = word_of(s >> 1, g) + (s & 1) * 8;
        return d >= (s >> 1) * 64 ? d : -1;
    }

    // The first and the last chunk (CH positions) of a span that hold
    // positions in sight.
    struct Ends {
        int32_t first, last;
    };

    // The position whose page chunk i of a tile lies in: a chunk never
    // crosses pages. Where none of its positions is in sight (their page may
    // be gone) the nearest that are stand in; they are masked.
    static __device__ __forceinline__ int32_t chunk_of(int32_t j0, int32_t i, const Ends &e)
    {
        const int32_t j = j0 + i * CH;
        const int32_t k = j < e.last ? j : e.last;
        return k > e.first ? k : e.first;
    }

    // Pages of a tile's positions, 16 by 16 (no page is shorter): read with
    // scalar loads, whose waits leave the vector loads in flight alone. A bad
    // one sets `bad` and stands as page 0.
    struct Pages {
        int32_t x, y, z, w;  // (the last two with 64-position tiles)
    };
    static __device__ __forceinline__ int32_t page_at(const BlockArgs &g, int32_t b, int32_t j,
                                                      const Ends &e, bool &bad)
    {
        typedef const __attribute__((address_space(4))) int32_t *Table;
        j = j < e.last ? j : e.last;
        j = (j > e.first ? j : e.first) >> g.page_shift;
        const bool in = j < g.table_stride;
        const int32_t id =
            ((Table)(uintptr_t)(g.table + (int64_t)b * g.table_stride))[in ? j : 0];
        const bool ok = in && (uint32_t)id < (uint64_t)g.n_pages;
        bad |= !ok;
        return ok ? id : 0;
    }
    static __device__ __forceinline__ Pages pages_of(const BlockArgs &g, int32_t b, int32_t j0,
                                                     const Ends &e, bool &bad)
    {
        Pages p;
        p.x = page_at(g, b, j0, e, bad);
        p.y = page_at(g, b, j0 + 16, e, bad);
        p.z = TK == 64 ? page_at(g, b, j0 + 32, e, bad) : 0;
        p.w = TK == 64 ? page_at(g, b, j0 + 48, e, bad) : 0;
        return p;
    }
    // the page of chunk i of a tile
    static __device__ __forceinline__ int32_t pick(const Pages &p, int i)
    {
        // (values, not lvalues: the struct must not be selected by address)
        const int32_t x = p.x, y = p.y, z = p.z, w = p.w;
        if constexpr (TK == 32)
            return (i & 2) ? y : x;
        const int32_t lo = (i & 1) ? y : x, hi = (i & 1) ? w : z;
        return (i & 2) ? hi : lo;
    }

    // Where this lane's K words of a tile start, for word 0 of block 0, dims
    // left out: row i of a 16-position block stands for position CH (i / 4) +
    // i % 4 (+ 4 for the second block, + 8 and 12 for the second step).
    static __device__ __forceinline__ const C *k_row(const C *kc, const Pages &p, int32_t j0,
                                                     const Ends &e, const BlockArgs &g, int32_t h,
                                                     int lane)
    {
        const int i = lane & 15;
        const int32_t tokens = 1 << g.page_shift, at = chunk_of(j0, i >> 2, e);
        return kc + (((int64_t)pick(p, i >> 2) * g.kv_heads + h) * tokens +
                     (at & (tokens - 1)) + (i & 3)) * D;
    }
    // Where this lane's V words of a tile start: dim lane % 16, + 16 a block.
    static __device__ __forceinline__ const C *v_row(const C *vc, const Pages &p, int32_t j0,
                                                     const Ends &e, const BlockArgs &g, int32_t h,
                                                     int lane)
    {
        const int32_t tokens = 1 << g.page_shift, at = chunk_of(j0, lane >> 4, e);
        return vc + (((int64_t)pick(p, lane >> 4) * g.kv_heads + h) * D + (lane & 15)) * tokens +
               (at & (tokens - 1));
    }

    // step s of a K block's words as a matrix operand
    static __device__ __forceinline__ U4 k_frag(const U4 (&k)[KW], int s)
    {
        if constexpr (kByte)
            return (s & 1) ? widen8<T>(k[s >> 1][2], k[s >> 1][3])
                           : widen8<T>(k[s >> 1][0], k[s >> 1][1]);
        else
            return k[s];
    }
    static __device__ __forceinline__ U4 v_frag(const U4 &v, int n)
    {
        if constexpr (kByte)
            return n ? widen8<T>(v[2], v[3]) : widen8<T>(v[0], v[1]);
        else
            return v;
    }

    // Step s of this lane's row m of the query rows as a matrix operand, zero
    // from row m1 on; `flip` turns the signs where the scale is negative.
    static __device__ __forceinline__ U4 q_frag(const AttendArgs &a, int32_t b, int32_t h,
                                                int32_t G, int32_t m, int32_t m1, int s, int grp,
                                                uint32_t flip)
    {
        const int d = dim_of(s, grp);
        if (m >= m1 || d < 0)
            return U4{0u, 0u, 0u, 0u};
        const int32_t t = m / G;
        return *(const U4 *)((const T *)a.q + ((int64_t)b * a.blk.rows + t) * a.q_stride +
                             (int64_t)(h * G + m - t * G) * D + d) ^
               flip;
    }

    // The last position in sight of a block's row t (a tree's: its node) and
    // the first; of a tree's row at most the one behind the root, since its
    // branch, which the window has cut already, says the rest.
    static __device__ __forceinline__ void sight_of_row(const AttendArgs &a, int32_t t,
                                                        int32_t root, const char *branches,
                                                        int32_t &pos, int32_t &low)
    {
        if constexpr (TREE) {
            pos = t;
            const int32_t at = a.window ? root + Branches::depth(branches, t) : 0;
            low = a.window && at >= a.window ? at - a.window + 1 : 0;
            low = low > root + 1 ? root + 1 : low;
        } else {
            pos = root + t;
            low = a.window && pos >= a.window ? pos - a.window + 1 : 0;
        }
    }

    // One block of query rows against one tile: masks the scores where the
    // tile reaches over an end of someone's sight, raises the running
    // maximum, turns the scores into probabilities (st) and operands (pf).
    static __device__ __forceinline__ void soften(F4 (&st)[2 * NB], U4 (&pf)[NB], float &m,
                                                  float &l, F4 (&o)[DB], float c, bool edge,
                                                  int32_t j, int32_t low, int32_t high,
                                                  uint32_t branch)
    {
        if (edge) {
#pragma unroll
            for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (j + t * 4 + r > high || j + t * 4 + r < low ||
                        (TREE && !((branch >> (t * 4 + r)) & 1)))
                        st[t][r] = -INFINITY;
        }
        float mx = fmaxf(fmaxf(st[0][0], st[0][1]), fmaxf(st[0][2], st[0][3]));
#pragma unroll
        for (int t = 1; t < 2 * NB; ++t)
            mx = fmaxf(mx, fmaxf(fmaxf(st[t][0], st[t][1]), fmaxf(st[t][2], st[t][3])));
        mx *= c;
        if (__any(mx > m + kSlack)) {
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float mn = fmaxf(m, mx);
            const float f = __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int i = 0; i < DB; ++i)
                o[i] *= f;
        }
        const float shift = kLift - m;
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                st[t][r] = __builtin_amdgcn_exp2f(fmaf(st[t][r], c, shift));
                l += st[t][r];
            }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            pf[nb] = U4{pack2<T>(st[2 * nb][0], st[2 * nb][1]),
                        pack2<T>(st[2 * nb][2], st[2 * nb][3]),
                        pack2<T>(st[2 * nb + 1][0], st[2 * nb + 1][1]),
                        pack2<T>(st[2 * nb + 1][2], st[2 * nb + 1][3])};
    }

    // NaN in query rows [m0, m1) of a request.
    static __device__ __forceinline__ void fill_nan(T *out, float *lse, const BlockArgs &g,
                                                    int32_t h, int32_t G, int32_t m0, int32_t m1)
    {
        for (int32_t i = threadIdx.x; i < (m1 - m0) * D; i += kWaves * kWave) {
            const int32_t r = m0 + i / D, t = r / G;
            out[((int64_t)t * g.q_heads + h * G + r - t * G) * D + i % D] = from_f32<T>(NAN);
        }
        for (int32_t r = m0 + threadIdx.x; lse && r < m1; r += kWaves * kWave)
            lse[(int64_t)(r / G) * g.q_heads + h * G + r % G] = NAN;
    }

    // An edge tile's V: positions past the span's end become zero, and so does
    // a position with an infinity or a NaN (0 times it would be NaN in the
    // rows that do not see it), whose share is then added to the rows that
    // do. `st` holds the probabilities.
    static __device__ __forceinline__ void hide(U4 (&v)[DB], F4 (&o)[MB][DB],
                                                const F4 (&st)[MB][2 * NB],
                                                const int32_t (&pos)[MB],
                                                const int32_t (&low)[MB], const C *vc, int32_t b,
                                                int32_t j0, int32_t s1, const BlockArgs &g,
                                                int32_t h, int lane, const char *branches,
                                                bool branchy, int32_t root)
    {
        const int grp = lane >> 4;
        const int32_t left = s1 - (j0 + grp * CH);  // slots 0..left are in the span
        constexpr int kPer = kByte ? 4 : 2;               // cells of a 32-bit word
        constexpr uint32_t kBits = kByte ? 0xffu : 0xffffu;
        // NaN (and infinity): all ones in the exponent (8-bit: in all but the sign)
        constexpr uint32_t kExp = kByte ? 0x7fu : (sizeof(typename Frag<T>::V2) == 4 &&
                                                           __is_same(T, __bf16)
                                                       ? 0x7f80u
                                                       : 0x7c00u);
        uint32_t odd = 0;  // slots with such a cell
#pragma unroll
        for (int e = 0; e < CH; ++e) {
            const uint32_t mask = kBits << (e % kPer * (32 / kPer));
            bool any = false;
#pragma unroll
            for (int i = 0; i < DB; ++i) {
                const uint32_t w = v[i][e / kPer] >> (e % kPer * (32 / kPer));
                any |= (w & kExp) == kExp;
            }
            any &= e <= left;
            const uint64_t vote = __ballot(any);
            if ((vote >> (grp * 16)) & 0xffffu)
                odd |= 1u << e;
            if (e > left || ((odd >> e) & 1)) {
#pragma unroll
                for (int i = 0; i < DB; ++i)
                    v[i][e / kPer] &= ~mask;
            }
        }
        if (!__any(odd != 0))
            return;
        const int32_t tokens = 1 << g.page_shift;
        for (int from = 0; from < 4; ++from) {
#pragma unroll
            for (int e = 0; e < CH; ++e) {
                if (!((__shfl(odd, from * 16) >> e) & 1))
                    continue;
                const int32_t j = j0 + from * CH + e;
                const int32_t page = page_of(g, b, j), id = page < 0 ? 0 : page;
                const C *p = vc + (((int64_t)id * g.kv_heads + h) * D + grp * 4) * tokens +
                             (j & (tokens - 1));
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    const float w = to_f32((T)__shfl(st[mb][e / 4][e % 4], from * 16 + (lane & 15)));
                    // (a tree's rows: pos is their node. Without branches nothing
                    // lies behind the root.)
                    const bool sees =
                        TREE ? !branchy || (Branches::bits(branches, pos[mb], j, root) & 1)
                             : j <= pos[mb];
                    if (sees && j >= low[mb]) {
#pragma unroll
                        for (int i = 0; i < DB; ++i)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                o[mb][i][r] += w * to_f32(p[(int64_t)(i * 16 + r) * tokens]);
                    }
                }
            }
        }
    }
};

// The share of a workgroup: query rows [m0, m1) of one request and kv head,
// positions [s0, s1].
struct Work {
    int32_t b, h, G, length, m0, m1, lo, s0, s1;
    int64_t at;   // its partial results' first row
    bool whole;   // the span is all the rows see: no partial results
};

// Finds it from the block index; false when there is none. A request with
// bad inputs is written here.
template <typename K, typename T, int M>
__device__ __forceinline__ bool work_of(const AttendArgs &a, const Split &sp, Work &w)
{
    const BlockArgs &g = a.blk;
    // Workgroups that read the same span (the tiles of query rows) are 8
    // apart: on one XCD, whose L2 then serves the span once. The kv heads of a
    // span, which lie in the same pages, come one after the other: 64 ragged
    // requests of 8 heads run at 5.1 TB/s so, at 4.1 with a head's spans first.
    uint32_t id = blockIdx.x;
    const uint32_t mt = id / 8 % sp.m_tiles;
    id = id / 8 / sp.m_tiles * 8 + id % 8;
    const uint32_t per = (uint32_t)g.kv_heads * sp.splits;
    if (id >= per * g.batch)
        return false;
    w.h = id % g.kv_heads;
    const int32_t split = id / g.kv_heads % sp.splits;
    w.b = id / per;
    w.G = g.q_heads / g.kv_heads;
    w.m0 = mt * M;
    uint32_t err;
    const int32_t n = block_rows(g, w.b, w.length, err);
    if (n < 0) {
        const int32_t end = g.rows * w.G;
        if (split == 0) {
            if (threadIdx.x == 0 && w.h == 0 && mt == 0)
                atomicOr(g.err, err);
            K::fill_nan((T *)a.out + (int64_t)w.b * g.rows * g.q_heads * g.head_dim,
                        a.out_lse ? a.out_lse + (int64_t)w.b * g.rows * g.q_heads : nullptr, g,
                        w.h, w.G, w.m0, w.m0 + M < end ? w.m0 + M : end);
        }
        return false;
    }
    if (w.m0 >= n * w.G)
        return false;
    w.m1 = w.m0 + M < n * w.G ? w.m0 + M : n * w.G;
    const Sight s = sight_of<K::TK, K::kTree>(a, w.length, w.m0 / w.G, (w.m1 - 1) / w.G);
    const int32_t span = span_of<K::kTree, K::kGrain>(sp, s);
    const int64_t s0 = s.start + (int64_t)split * span;
    if (s0 > s.hi)
        return false;
    w.s0 = (int32_t)s0;
    w.s1 = span <= s.hi - w.s0 ? w.s0 + span - 1 : s.hi;
    w.lo = s.lo;
    w.whole = span > s.hi - s.start;
    w.at = (((int64_t)w.b * g.kv_heads + w.h) * sp.splits + split) * (sp.m_tiles * (int64_t)M);
    return true;
}

// A workgroup that met a bad page, or parent: its rows, or its partial
// results, are NaN.
template <typename K, typename T, int D>
__device__ __forceinline__ void give_up(const AttendArgs &a, const Split &sp, const Work &w,
                                        uint32_t err)
{
    const BlockArgs &g = a.blk;
    if (threadIdx.x == 0)
        atomicOr(g.err, err);
    if (w.whole) {
        K::fill_nan((T *)a.out + (int64_t)w.b * g.rows * g.q_heads * D,
                    a.out_lse ? a.out_lse + (int64_t)w.b * g.rows * g.q_heads : nullptr, g, w.h,
                    w.G, w.m0, w.m1);
        return;
    }
    for (int32_t r = w.m0 + threadIdx.x; r < w.m1; r += kWaves * kWave)
        sp.ml[w.at + r] = float2{0.0f, NAN};
    for (int32_t i = threadIdx.x; i < (w.m1 - w.m0) * D; i += kWaves * kWave)
        sp.o[(w.at + w.m0) * D + i] = NAN;
}

// Stores block i (16 dims) of query row `row`: y holds 4 of its dims.
template <typename T, int D>
__device__ __forceinline__ void store(const AttendArgs &a, const Split &sp, const Work &w,
                                      int32_t row, int i, int grp, F4 y, float inv)
{
    if (w.whole) {
        const int32_t t = row / w.G, hd = w.h * w.G + row - t * w.G;
        y *= inv;
        *(U2 *)((T *)a.out + (((int64_t)w.b * a.blk.rows + t) * a.blk.q_heads + hd) * D + i * 16 +
                grp * 4) = U2{pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3])};
    } else {
        *(F4 *)(sp.o + (w.at + row) * D + i * 16 + grp * 4) = y;
    }
}

__device__ __forceinline__ void store_ml(const AttendArgs &a, const Split &sp, const Work &w,
                                         int32_t row, float m, float l)
{
    if (!w.whole) {
        sp.ml[w.at + row] = float2{m, l};
    } else if (a.out_lse) {
        const int32_t t = row / w.G, hd = w.h * w.G + row - t * w.G;
        a.out_lse[((int64_t)w.b * a.blk.rows + t) * a.blk.q_heads + hd] =
            (m - kLift) * kLn2 + __logf(l);
    }
}

// Up to 32 query rows: every wavefront holds all of them and takes tiles of
// its own in turn; K and V go from HBM into its registers. Bound by HBM: 64
// requests of 8,192 to 65,536 positions, 8 kv heads of 128 dims, one row of 4
// query heads a kv head: 1.75 to 1.89 ms over six runs, 5.1 to 5.5 TB/s of bf16
// cache (a plain streaming read reaches 6.3).
template <typename T, typename C, int D, int MB, bool TREE>
struct Narrow : Tiles<T, C, D, MB, TREE> {
    typedef Tiles<T, C, D, MB, TREE> S;
    static constexpr int TK = S::TK, NB = S::NB, DB = S::DB, KW = S::KW, KS = S::KS, CH = S::CH;
    static constexpr int M = 16 * MB;
    // (the join's sums lie over the query rows and the branches)
    static constexpr int kBranches = MB * KS * kWave * 16;
    static constexpr int kAcc = kWaves * 16 * D * 4, kQ = kBranches + (TREE ? Branches::kLds : 0);
    static constexpr int kLds = kAcc > kQ ? kAcc : kQ;

    static __device__ __forceinline__ void load_k(U4 (&k)[2 * NB][KW], const C *row, int grp)
    {
#pragma unroll
        for (int b = 0; b < 2 * NB; ++b)
#pragma unroll
            for (int w = 0; w < KW; ++w)
                k[b][w] = *(const U4 *)(row + b * 4 * D + S::word_of(w, grp));
    }
    // (A 128-byte line of a V row in a page of 64 positions or more serves two
    // tiles: a non-temporal load would fetch it twice, 4.3 against 5.7 TB/s.)
    static __device__ __forceinline__ void load_v(U4 (&v)[DB], const C *row, int32_t tokens)
    {
#pragma unroll
        for (int i = 0; i < DB; ++i)
            v[i] = *(const U4 *)(row + (int64_t)i * 16 * tokens);
    }

    static __device__ __forceinline__ void run(const AttendArgs &a, const Split &sp, char *lds,
                                               float2 *lds_ml)
    {
        const BlockArgs &g = a.blk;
        const int lane = threadIdx.x & (kWave - 1);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        const int grp = lane >> 4, col = lane & 15;
        Work w;
        if (!work_of<Narrow, T, M>(a, sp, w))
            return;
        const typename S::Ends ends{(w.lo > w.s0 ? w.lo : w.s0) / CH * CH, w.s1 / CH * CH};
        const int32_t tokens = 1 << g.page_shift;
        const C *kc = (const C *)a.k_cache, *vc = (const C *)a.v_cache;
        const int32_t root = w.length - 1;
        const bool branchy = TREE && (w.s1 > root || a.window);
        int32_t up = 0;
        bool stray = false;
        if (branchy)
            up = parent_of(a.parent, g, w.b, threadIdx.x, stray);
        // K of the next tile is on its way while this one's softmax and V^T P^T
        // run, V of the next while its K Q^T runs, page ids a tile earlier
        U4 k[2 * NB][KW], v[DB];
        bool bad = false;
        typename S::Pages pn{};
        int32_t j0 = w.s0 + wave * TK;
        if (j0 <= w.s1) {
            const typename S::Pages p = S::pages_of(g, w.b, j0, ends, bad);
            load_k(k, S::k_row(kc, p, j0, ends, g, w.h, lane), grp);
            load_v(v, S::v_row(vc, p, j0, ends, g, w.h, lane), tokens);
            pn = S::pages_of(g, w.b, j0 + kWaves * TK, ends, bad);
        }

        // the query rows as operands
        const float ks = g.k_scale ? g.k_scale[w.h] : 1.0f;
        const float c0 = a.scale * ks * kLog2e;
        const float c = factor(c0);
        const uint32_t flip = c0 < 0.0f ? 0x80008000u : 0u;
        U4 *qf = (U4 *)lds;
        U4 q1[MB == 1 ? KS : 1];
        if constexpr (MB == 1) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
                q1[i] = S::q_frag(a, w.b, w.h, w.G, w.m0 + col, w.m1, i, grp, flip);
        } else {
            for (int f = wave; f < MB * KS; f += kWaves)
                qf[f * kWave + lane] = S::q_frag(a, w.b, w.h, w.G, w.m0 + f / KS * 16 + col, w.m1,
                                                 f % KS, grp, flip);
            __syncthreads();
        }

        const char *const branches = lds + kBranches;
        if (branchy) {
            if (__syncthreads_or(stray)) {
                give_up<Narrow, T, D>(a, sp, w, kErrBlock);
                return;
            }
            Branches::build(lds + kBranches, up, g.draft_len[w.b] + 1, a.window);
        }

        // this lane's query rows: last (a tree's: node) and first position in
        // sight
        int32_t pos[MB], low[MB];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const int32_t r = w.m0 + mb * 16 + col, t = (r < w.m1 ? r : w.m1 - 1) / w.G;
            S::sight_of_row(a, t, root, branches, pos[mb], low[mb]);
        }
        const int32_t all_to = w.length - 1 + (TREE ? 0 : w.m0 / w.G);
        const int32_t end = w.length - 1 + (w.m1 - 1) / w.G;
        const int32_t all_from = a.window && end >= a.window ? end - a.window + 1 : 0;
        float m[MB], l[MB];
        F4 o[MB][DB];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            m[mb] = -FLT_MAX;
            l[mb] = 0.0f;
#pragma unroll
            for (int i = 0; i < DB; ++i)
                o[mb][i] = F4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        while (j0 <= w.s1) {
            const int32_t next = j0 + kWaves * TK;
            const bool edge = j0 < all_from || j0 + TK - 1 > all_to || j0 + TK - 1 > w.s1;
            F4 st[MB][2 * NB];
#pragma unroll
            for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    st[mb][t] = F4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < KS; ++i)
                        st[mb][t] = Frag<T>::mma(S::k_frag(k[t], i),
                                                 MB == 1 ? q1[i] : qf[(mb * KS + i) * kWave + lane],
                                                 st[mb][t]);
                }
            const typename S::Pages p = pn;
            if (next <= w.s1) {
                load_k(k, S::k_row(kc, p, next, ends, g, w.h, lane), grp);
                pn = S::pages_of(g, w.b, next + kWaves * TK, ends, bad);
            }
            U4 pf[MB][NB];
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                S::soften(st[mb], pf[mb], m[mb], l[mb], o[mb], c, edge, j0 + grp * CH, low[mb],
                          TREE || pos[mb] > w.s1 ? w.s1 : pos[mb],
                          TREE && edge && branchy
                              ? Branches::bits(branches, pos[mb], j0 + grp * CH, root)
                              : 0xffffffffu);
            if (edge)
                S::hide(v, o, st, pos, low, vc, w.b, j0, w.s1, g, w.h, lane, branches, branchy,
                        root);
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const U4 vf = S::v_frag(v[i], nb);
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
                        o[mb][i] = Frag<T>::mma(vf, pf[mb][nb], o[mb][i]);
                }
            if (next <= w.s1)
                load_v(v, S::v_row(vc, p, next, ends, g, w.h, lane), tokens);
            j0 = next;
        }

        // join the wavefronts: common maxima, then each sums a share of the dims
        const float vs = g.v_scale ? g.v_scale[w.h] : 1.0f;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            l[mb] += __shfl_xor(l[mb], 16);
            l[mb] += __shfl_xor(l[mb], 32);
            if (grp == 0)
                lds_ml[wave * M + mb * 16 + col] = float2{m[mb], l[mb]};
        }
        // (also: every wavefront is done with qf)
        if (__syncthreads_or(bad)) {
            give_up<Narrow, T, D>(a, sp, w, kErrPage);
            return;
        }
        F4 *acc = (F4 *)lds;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            float top = -FLT_MAX, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kWaves; ++i)
                top = fmaxf(top, lds_ml[i * M + mb * 16 + col].x);
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                const float2 y = lds_ml[i * M + mb * 16 + col];
                sum += y.y * __builtin_amdgcn_exp2f(y.x - top);
            }
            const float f = __builtin_amdgcn_exp2f(m[mb] - top) * vs;
            if (mb > 0)
                __syncthreads();
#pragma unroll
            for (int i = 0; i < DB; ++i)
                acc[(wave * DB + i) * kWave + lane] = o[mb][i] * f;
            __syncthreads();
            const int32_t row = w.m0 + mb * 16 + col;
            const float inv = 1.0f / sum;
            for (int i = wave; i < DB; i += kWaves) {
                F4 y = acc[i * kWave + lane];
#pragma unroll
                for (int n = 1; n < kWaves; ++n)
                    y += acc[(n * DB + i) * kWave + lane];
                if (row < w.m1)
                    store<T, D>(a, sp, w, row, i, grp, y, inv);
            }
            if (row < w.m1 && wave == 0 && grp == 0)
                store_ml(a, sp, w, row, top, sum);
        }
    }
};

template <typename T, typename C, int D, int MB, bool TREE>
__global__ __launch_bounds__(kWaves *kWave, D <= 128 ? 2 : 1) void attend_narrow(AttendArgs a,
                                                                                 Split sp)
{
    typedef Narrow<T, C, D, MB, TREE> K;
    __shared__ __attribute__((aligned(16))) char lds[K::kLds];
    __shared__ float2 lds_ml[kWaves * K::M];
    K::run(a, sp, lds, lds_ml);
}

// More query rows: each wavefront holds a quarter of them (RB blocks of 16),
// and all four work on the same tile, which goes from HBM straight into LDS
// (direct loads, in the order of the matrix operands: 1 KB each, read back
// lane by lane). A ring of kStages tiles is in flight; one barrier a tile.
// Bound by HBM with matrix and vector work in half of the cycles: 16 requests
// of 262,144 positions, 2 kv heads of 128 dims, 128 query rows each: 0.88 to 0.95
// ms over six runs, 4.5 to 4.9 TB/s, 578 to 627 TFLOP/s; 2.00 ms when every
// wavefront held 64 rows and the cache was read by two workgroups.
template <typename T, typename C, int D, int RB, bool TREE>
struct Wide : Tiles<T, C, D, RB, TREE> {
    typedef Tiles<T, C, D, RB, TREE> S;
    static constexpr int TK = S::TK, NB = S::NB, DB = S::DB, KW = S::KW, KS = S::KS, CH = S::CH;
    static constexpr int M = 16 * RB * kWaves;
    static constexpr int FK = 2 * NB * KW;                        // K words of a tile, a lane
    static constexpr int kLoads = (FK + DB + kWaves - 1) / kWaves;  // of a wavefront, a tile
    static constexpr int kStage = kLoads * kWaves * 1024;
    static constexpr int kFit = 65536 / kStage;
    static constexpr int kStages = kFit < 2 ? 2 : (kFit > 6 ? 6 : kFit);
    static constexpr int kBranches = kStages * kStage;
    static constexpr int kLds = kBranches + (TREE ? Branches::kLds : 0);
    static_assert(kBranches <= 65536, "M0 holds 16 bits of an LDS address");

    static __device__ __forceinline__ void run(const AttendArgs &a, const Split &sp, char *lds)
    {
        const BlockArgs &g = a.blk;
        const int lane = threadIdx.x & (kWave - 1);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        const int grp = lane >> 4, col = lane & 15;
        Work w;
        if (!work_of<Wide, T, M>(a, sp, w))
            return;
        const typename S::Ends ends{(w.lo > w.s0 ? w.lo : w.s0) / CH * CH, w.s1 / CH * CH};
        const int32_t tokens = 1 << g.page_shift;
        const C *kc = (const C *)a.k_cache, *vc = (const C *)a.v_cache;
        bool bad = false;
        const int32_t root = w.length - 1;
        const bool branchy = TREE && (w.s1 > root || a.window);
        int32_t up = 0;
        bool stray = false;
        if (branchy)
            up = parent_of(a.parent, g, w.b, threadIdx.x, stray);

        // load n of this wavefront brings operand f = 4 n + wave of a tile:
        // first K's words, block by block, then V's, then (to fill up) V's
        // first again
        const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
        const auto fetch = [&](int32_t j0, const typename S::Pages &p, int slot) {
            const C *kr = S::k_row(kc, p, j0, ends, g, w.h, lane);
            const C *vr = S::v_row(vc, p, j0, ends, g, w.h, lane);
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                const int f = n * kWaves + wave;
                const C *from;
                if (f < FK)
                    from = kr + f / KW * 4 * D + S::word_of(f % KW, grp);
                else
                    from = vr + (int64_t)(f - FK < DB ? f - FK : 0) * 16 * tokens;
                const uint32_t to =
                    __builtin_amdgcn_readfirstlane(ring + slot * kStage + f * 1024);
                // (M0, the LDS address, is the compiler's: put back; a load may
                // not follow its write at once)
                uint32_t m0;
                asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\t"
                             "global_load_lds_dwordx4 %1, off\n\ts_mov_b32 m0, %0"
                             : "=&s"(m0)
                             : "v"(from), "s"(to)
                             : "memory");
            }
        };
        const int32_t tiles = (w.s1 - w.s0) / TK + 1;
        typename S::Pages pn = S::pages_of(g, w.b, w.s0, ends, bad);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            if (i < tiles)
                fetch(w.s0 + i * TK, pn, i);
            pn = S::pages_of(g, w.b, w.s0 + (i + 1) * TK, ends, bad);
        }

        const float ks = g.k_scale ? g.k_scale[w.h] : 1.0f;
        const float c0 = a.scale * ks * kLog2e;
        const float c = factor(c0);
        const uint32_t flip = c0 < 0.0f ? 0x80008000u : 0u;
        const char *const branches = lds + kBranches;
        if (branchy) {
            if (__syncthreads_or(stray)) {
                // (its LDS is another workgroup's once this one ends)
                asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
                give_up<Wide, T, D>(a, sp, w, kErrBlock);
                return;
            }
            Branches::build(lds + kBranches, up, g.draft_len[w.b] + 1, a.window);
        }
        U4 q[RB][KS];
        int32_t pos[RB], low[RB];
        float m[RB], l[RB];
        F4 o[RB][DB];
        const int32_t mine = w.m0 + wave * 16 * RB;
#pragma unroll
        for (int mb = 0; mb < RB; ++mb) {
            const int32_t r = mine + mb * 16 + col;
            S::sight_of_row(a, (r < w.m1 ? r : w.m1 - 1) / w.G, root, branches, pos[mb], low[mb]);
            m[mb] = -FLT_MAX;
            l[mb] = 0.0f;
#pragma unroll
            for (int i = 0; i < KS; ++i)
                q[mb][i] = S::q_frag(a, w.b, w.h, w.G, r, w.m1, i, grp, flip);
#pragma unroll
            for (int i = 0; i < DB; ++i)
                o[mb][i] = F4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const int32_t all_to = w.length - 1 + (TREE ? 0 : w.m0 / w.G);
        const int32_t end = w.length - 1 + (w.m1 - 1) / w.G;
        const int32_t all_from = a.window && end >= a.window ? end - a.window + 1 : 0;

        int slot = 0;
        for (int32_t i = 0; i < tiles; ++i) {
            const int32_t j0 = w.s0 + i * TK;
            // This wavefront's loads of tile i are done when at most those of
            // the kStages - 2 tiles behind it are in flight (near the end
            // there are fewer: wait for all); the barrier then stands for the
            // other wavefronts' loads, and for their reads of the slot that
            // the next fetch overwrites.
            if (i + kStages - 2 < tiles)
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier"
                             :
                             : "n"(kLoads *(kStages - 2))
                             : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : : : "memory");
            const int32_t ahead = i + kStages - 1;
            if (ahead < tiles) {
                fetch(w.s0 + ahead * TK, pn, slot == 0 ? kStages - 1 : slot - 1);
                pn = S::pages_of(g, w.b, w.s0 + (ahead + 1) * TK, ends, bad);
            }
            const U4 *x = (const U4 *)(lds + slot * kStage) + lane;
            slot = slot + 1 == kStages ? 0 : slot + 1;
            const bool edge = j0 < all_from || j0 + TK - 1 > all_to || j0 + TK - 1 > w.s1;
            F4 st[RB][2 * NB];
#pragma unroll
            for (int t = 0; t < 2 * NB; ++t) {
                U4 k[KW];
#pragma unroll
                for (int n = 0; n < KW; ++n)
                    k[n] = x[(t * KW + n) * kWave];
#pragma unroll
                for (int mb = 0; mb < RB; ++mb) {
                    st[mb][t] = F4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int n = 0; n < KS; ++n)
                        st[mb][t] = Frag<T>::mma(S::k_frag(k, n), q[mb][n], st[mb][t]);
                }
            }
            U4 pf[RB][NB];
#pragma unroll
            for (int mb = 0; mb < RB; ++mb)
                S::soften(st[mb], pf[mb], m[mb], l[mb], o[mb], c, edge, j0 + grp * CH, low[mb],
                          TREE || pos[mb] > w.s1 ? w.s1 : pos[mb],
                          TREE && edge && branchy
                              ? Branches::bits(branches, pos[mb], j0 + grp * CH, root)
                              : 0xffffffffu);
            U4 v[DB];
#pragma unroll
            for (int n = 0; n < DB; ++n)
                v[n] = x[(FK + n) * kWave];
            if (edge)
                S::hide(v, o, st, pos, low, vc, w.b, j0, w.s1, g, w.h, lane, branches, branchy,
                        root);
#pragma unroll
            for (int n = 0; n < DB; ++n)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const U4 vf = S::v_frag(v[n], nb);
#pragma unroll
                    for (int mb = 0; mb < RB; ++mb)
                        o[mb][n] = Frag<T>::mma(vf, pf[mb][nb], o[mb][n]);
                }
        }

        if (bad) {  // the same on every wavefront: they went through the same tiles
            give_up<Wide, T, D>(a, sp, w, kErrPage);
            return;
        }
        const float vs = g.v_scale ? g.v_scale[w.h] : 1.0f;
#pragma unroll
        for (int mb = 0; mb < RB; ++mb) {
            l[mb] += __shfl_xor(l[mb], 16);
            l[mb] += __shfl_xor(l[mb], 32);
            const int32_t row = mine + mb * 16 + col;
            if (row >= w.m1)
                continue;
            const float inv = 1.0f / l[mb];
#pragma unroll
            for (int i = 0; i < DB; ++i)
                store<T, D>(a, sp, w, row, i, grp, o[mb][i] * vs, inv);
            if (grp == 0)
                store_ml(a, sp, w, row, m[mb], l[mb]);
        }
    }
};

template <typename T, typename C, int D, int RB, bool TREE>
__global__ __launch_bounds__(kWaves *kWave, D <= 128 ? 2 : 1) void attend_wide(AttendArgs a,
                                                                               Split sp)
{
    typedef Wide<T, C, D, RB, TREE> K;
    __shared__ __attribute__((aligned(1024))) char lds[K::kLds];
    K::run(a, sp, lds);
}

// Joins the spans of a row: one wavefront per (request, row, query head). A
// lane takes 4 dims of every 256 / D'th span (D' = D up to a power of two);
// 8 loads are in flight, since a span's partial results are a round trip to
// L2 away and the launch is short.
template <typename T, int D, int TK, int M, bool TREE, int GRAIN>
__global__ __launch_bounds__(kWave) void join_kernel(AttendArgs a, Split sp)
{
    constexpr int kLanes = D <= 64 ? 16 : (D <= 128 ? 32 : 64);  // of a span
    constexpr int kSide = kWave / kLanes;                        // spans side by side
    constexpr int kDeep = 8;
    const BlockArgs &g = a.blk;
    const int32_t lane = threadIdx.x, hd = blockIdx.x % (uint32_t)g.q_heads;
    const uint32_t bt = blockIdx.x / (uint32_t)g.q_heads;
    const int32_t t = bt % (uint32_t)g.rows, b = bt / (uint32_t)g.rows;
    int32_t length;
    uint32_t err;
    const int32_t n = block_rows(g, b, length, err);
    if (t >= n)
        return;
    const int32_t G = g.q_heads / g.kv_heads, h = hd / G;
    const int32_t row = t * G + hd - h * G, m0 = row / M * M;
    const int32_t m1 = m0 + M < n * G ? m0 + M : n * G;
    const Sight s = sight_of<TK, TREE>(a, length, m0 / G, (m1 - 1) / G);
    const int32_t spans = (s.hi - s.start) / span_of<TREE, GRAIN>(sp, s) + 1;
    if (spans == 1)
        return;
    const int64_t rows = (int64_t)sp.m_tiles * M;
    const int64_t at = ((int64_t)b * g.kv_heads + h) * sp.splits * rows + row;
    const int d = lane % kLanes * 4, side = lane / kLanes;
    float top = -FLT_MAX, sum = 0.0f;
    F4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int32_t base = 0; base < spans; base += kWave) {
        const int32_t count = spans - base < kWave ? spans - base : kWave;
        const float2 v = lane < count ? sp.ml[at + (base + lane) * rows] : float2{-FLT_MAX, 0.0f};
        float mx = v.x;
        for (int i = kWave / 2; i; i >>= 1)
            mx = fmaxf(mx, __shfl_xor(mx, i));
        mx = fmaxf(mx, top);
        const float old = __builtin_amdgcn_exp2f(top - mx);
        top = mx;
        const float f = __builtin_amdgcn_exp2f(v.x - top);
        float part = v.y * f;
        for (int i = kWave / 2; i; i >>= 1)
            part += __shfl_xor(part, i);
        sum = sum * old + part;
        y *= old;
        for (int32_t i = 0; i < count; i += kDeep * kSide) {
            F4 x[kDeep];
            float w[kDeep];
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                const int32_t k = i + u * kSide + side;
                w[u] = __shfl(f, k & (kWave - 1));
                x[u] = F4{0.0f, 0.0f, 0.0f, 0.0f};
                if (k < count && d < D)
                    x[u] = *(const F4 *)(sp.o + (at + (base + k) * rows) * D + d);
            }
#pragma unroll
            for (int u = 0; u < kDeep; ++u)
                y += x[u] * w[u];
        }
    }
#pragma unroll
    for (int i = kLanes; i < kWave; i <<= 1)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            y[r] += __shfl_xor(y[r], i);
    const int64_t r = ((int64_t)b * g.rows + t) * g.q_heads + hd;
    if (side == 0 && d < D)
        *(U2 *)((T *)a.out + r * D + d) =
            U2{pack2<T>(y[0] / sum, y[1] / sum), pack2<T>(y[2] / sum, y[3] / sum)};
    if (a.out_lse && lane == 0)
        a.out_lse[r] = (top - kLift) * kLn2 + __logf(sum);
}

}  // namespace

}  // namespace pld
