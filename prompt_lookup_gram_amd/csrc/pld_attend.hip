// Attention of the verify block's rows over the paged cache, for gfx950
// (MI355X).
//
// Mathematics. A workgroup takes one request, one kv head, up to 16 MB query
// rows (row m = block row t, query head g of the group: m = t * G + g) and a
// span of positions; its wavefronts take tiles of the span in turn, each
// with its own running maximum m, sum l and output O (one pass, no tile is
// read twice):
//   S^T = K Q^T,  P^T = 2^(c S^T - m + kLift),  O^T += V^T P^T,  l += sum P,
// c = scale * log2 e. Both products are 16x16x32 matrix instructions whose
// left operand is the cache as it lies in memory: a lane holds 16 bytes of a
// K row (positions x dims) or of a V row (dims x positions; that is why V
// pages hold positions side by side), so K and V go from HBM into registers
// with no LDS and no transpose. The result layout of S^T (lane: one query
// row, positions 4 (lane / 16) + r) is the right operand's layout of P^T once
// the positions of a tile are dealt to the K rows in the matching order,
// so P never leaves its lane either.
//
// m is raised only when a score passes it by kSlack (the sum and O are then
// rescaled); P is lifted by 2^kLift, so that in fp16 probabilities down to
// 2^-26 of the row's largest keep all their bits and 2^(kLift + kSlack) stays
// below 65504.

#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

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

// How a launch splits the positions: spans of `span` positions (a multiple
// of the tile), `splits` of them at most; partial results of a request whose
// positions take more than one.
struct Split {
    int32_t span;
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

template <int TK>
__device__ __forceinline__ Sight sight_of(const AttendArgs &a, int32_t length, int32_t t0,
                                          int32_t t1)
{
    Sight s;
    const int32_t first = length - 1 + t0;
    s.lo = a.window && first >= a.window ? first - a.window + 1 : 0;
    s.hi = length - 1 + t1;
    s.start = s.lo / TK * TK;
    return s;
}

template <typename T, typename C, int D, int MB>
struct Kernel {
    static constexpr bool kByte = sizeof(C) == 1;
    static constexpr int TK = kByte ? 64 : 32;  // positions of a tile
    static constexpr int NB = TK / 32;          // 32-position steps of V^T P^T
    static constexpr int KS = D / 32;           // steps of K Q^T
    static constexpr int DB = D / 16;           // blocks of 16 dims
    static constexpr int KW = kByte ? (KS + 1) / 2 : KS;  // 16-byte words of a K row, a lane
    static constexpr int M = 16 * MB;
    static constexpr int kLds = kWaves * 16 * D * 4 > M * D * 2 ? kWaves * 16 * D * 4 : M * D * 2;

    // The dims of step s that lane group g holds start here: with 8-bit cells
    // a lane's 16 bytes serve two steps.
    static __device__ __forceinline__ int dim_of(int s, int g)
    {
        if (kByte && (s | 1) < KS)
            return (s >> 1) * 64 + g * 16 + (s & 1) * 8;
        return s * 32 + g * 8;
    }

    struct Tile {
        U4 k[2 * NB][KW];
        U4 v[DB];
    };

    // The first and the last chunk (8 NB positions) of a span that hold
    // positions in sight.
    struct Ends {
        int32_t first, last;
    };

    // The position whose page a lane's cells of a tile lie in, for K row
    // block i / 4 or V lane group i: 8 NB positions, inside one page. Where
    // none of them is in sight (their page may be gone) the nearest that are
    // stand in; they are masked.
    static __device__ __forceinline__ int32_t chunk_of(int32_t j0, int32_t i, const Ends &e)
    {
        const int32_t j = j0 + i * (8 * NB);
        const int32_t k = j < e.last ? j : e.last;
        return k > e.first ? k : e.first;
    }

    // Pages of a tile's K rows and V columns for this lane; a bad one sets
    // `bad` and stands as page 0.
    struct Pages {
        int32_t k, v;
    };
    static __device__ __forceinline__ Pages pages_of(const BlockArgs &g, int32_t b, int32_t j0,
                                                     const Ends &e, int lane, bool &bad)
    {
        Pages p;
        p.k = page_of(g, b, chunk_of(j0, (lane & 15) >> 2, e));
        p.v = page_of(g, b, chunk_of(j0, lane >> 4, e));
        bad |= (p.k | p.v) < 0;
        p.k = p.k < 0 ? 0 : p.k;
        p.v = p.v < 0 ? 0 : p.v;
        return p;
    }

    static __device__ __forceinline__ void load_k(Tile &x, const C *kc, int32_t page, int32_t j0,
                                                  const Ends &e, const BlockArgs &g, int32_t h,
                                                  int lane)
    {
        const int grp = lane >> 4;
        const int32_t tokens = 1 << g.page_shift;
        // row i of a 16-position block stands for position 8 NB (i / 4) + i % 4
        // (+ 4 for the second block, + 8 for the second step)
        const int i = lane & 15;
        const int32_t at = chunk_of(j0, i >> 2, e);
        const C *row = kc + (((int64_t)page * g.kv_heads + h) * tokens + (at & (tokens - 1)) +
                             (i & 3)) * D;
#pragma unroll
        for (int b = 0; b < 2 * NB; ++b) {
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const C *p = row + b * 4 * D;
                if constexpr (kByte) {
                    if (2 * w + 1 < KS)
                        x.k[b][w] = *(const U4 *)(p + w * 64 + grp * 16);
                    else {
                        const U2 y = *(const U2 *)(p + w * 64 + grp * 8);
                        x.k[b][w] = U4{y[0], y[1], 0u, 0u};
                    }
                } else {
                    x.k[b][w] = *(const U4 *)(p + w * 32 + grp * 8);
                }
            }
        }
    }

    static __device__ __forceinline__ void load_v(Tile &x, const C *vc, int32_t page, int32_t j0,
                                                  const Ends &e, const BlockArgs &g, int32_t h,
                                                  int lane)
    {
        const int32_t tokens = 1 << g.page_shift;
        const int32_t at = chunk_of(j0, lane >> 4, e);
        const C *p = vc + (((int64_t)page * g.kv_heads + h) * D + (lane & 15)) * tokens +
                     (at & (tokens - 1));
#pragma unroll
        for (int i = 0; i < DB; ++i)
            x.v[i] = *(const U4 *)(p + (int64_t)i * 16 * tokens);
    }

    // step s of K block b as a matrix operand
    static __device__ __forceinline__ U4 k_frag(const Tile &x, int b, int s)
    {
        if constexpr (kByte) {
            const U4 w = x.k[b][s >> 1];
            return (s & 1) ? widen8<T>(w[2], w[3]) : widen8<T>(w[0], w[1]);
        } else {
            return x.k[b][s];
        }
    }
    static __device__ __forceinline__ U4 v_frag(const Tile &x, int i, int n)
    {
        if constexpr (kByte)
            return n ? widen8<T>(x.v[i][2], x.v[i][3]) : widen8<T>(x.v[i][0], x.v[i][1]);
        else
            return x.v[i];
    }

    static __device__ void run(const AttendArgs &a, const Split &sp, char *lds, float2 *lds_ml)
    {
        const BlockArgs &g = a.blk;
        const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
        const int grp = lane >> 4, col = lane & 15;
        // workgroups that read the same span (the tiles of query rows) are 8
        // apart: on one XCD, whose L2 then serves the span once
        uint32_t id = blockIdx.x;
        const uint32_t mt = id / 8 % sp.m_tiles;
        id = id / 8 / sp.m_tiles * 8 + id % 8;
        const uint32_t per = (uint32_t)g.kv_heads * sp.splits;
        if (id >= per * g.batch)
            return;
        const int32_t b = id / per, h = id % per / sp.splits, split = id % sp.splits;
        const int32_t G = g.q_heads / g.kv_heads;
        const int32_t m0 = mt * M;
        int32_t length;
        uint32_t err;
        const int32_t n = block_rows(g, b, length, err);
        T *out = (T *)a.out + (int64_t)b * g.rows * g.q_heads * D;
        float *lse = a.out_lse ? a.out_lse + (int64_t)b * g.rows * g.q_heads : nullptr;
        if (n < 0) {
            if (split == 0) {
                if (threadIdx.x == 0 && h == 0 && mt == 0)
                    atomicOr(g.err, err);
                fill_nan(out, lse, g, h, G, m0, g.rows * G);
            }
            return;
        }
        if (m0 >= n * G)
            return;
        const int32_t m1 = m0 + M < n * G ? m0 + M : n * G;  // one past the last row
        const Sight s = sight_of<TK>(a, length, m0 / G, (m1 - 1) / G);
        const int32_t s0 = s.start + split * sp.span;
        if (s0 > s.hi)
            return;
        const int32_t s1 = sp.span <= s.hi - s0 ? s0 + sp.span - 1 : s.hi;  // inclusive
        const bool whole = sp.span > s.hi - s.start;  // this span is all of it

        // the query rows as operands
        U4 *qf = (U4 *)lds;
        const float ks = g.k_scale ? g.k_scale[h] : 1.0f;
        const float c0 = a.scale * ks * kLog2e;
        const float c = fabsf(c0);
        const uint32_t flip = c0 < 0.0f ? 0x80008000u : 0u;
        for (int f = wave; f < MB * KS; f += kWaves) {
            const int32_t m = m0 + f / KS * 16 + col;
            U4 x = {0u, 0u, 0u, 0u};
            if (m < m1) {
                const int32_t t = m / G;
                x = *(const U4 *)((const T *)a.q + ((int64_t)b * g.rows + t) * a.q_stride +
                                  (int64_t)(h * G + m - t * G) * D + dim_of(f % KS, grp));
            }
            qf[f * kWave + lane] = x ^ flip;
        }
        __syncthreads();

        // this lane's query rows: position and first position in sight
        int32_t pos[MB], low[MB];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const int32_t m = m0 + mb * 16 + col;
            pos[mb] = length - 1 + (m < m1 ? m : m1 - 1) / G;
            low[mb] = a.window && pos[mb] >= a.window ? pos[mb] - a.window + 1 : 0;
        }
        const int32_t pos_min = length - 1 + m0 / G;
        const int32_t low_max = a.window && s.hi >= a.window ? s.hi - a.window + 1 : 0;

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
        U4 q1[MB == 1 ? KS : 1];
        if constexpr (MB == 1) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
                q1[i] = qf[i * kWave + lane];
        }
        const C *kc = (const C *)a.k_cache, *vc = (const C *)a.v_cache;
        // K of the next tile is on its way while this one's softmax and V^T P^T
        // run, V of the next while its K Q^T runs, page ids a tile earlier
        Tile x;
        bool bad = false;
        Pages pg{0, 0}, pn{0, 0};
        const Ends ends{(s.lo > s0 ? s.lo : s0) / (8 * NB) * (8 * NB), s1 / (8 * NB) * (8 * NB)};
        int32_t j0 = s0 + wave * TK;
        if (j0 <= s1) {
            pg = pages_of(g, b, j0, ends, lane, bad);
            load_k(x, kc, pg.k, j0, ends, g, h, lane);
            load_v(x, vc, pg.v, j0, ends, g, h, lane);
            if (j0 + kWaves * TK <= s1)
                pn = pages_of(g, b, j0 + kWaves * TK, ends, lane, bad);
        }
        for (; j0 <= s1; j0 += kWaves * TK) {
            const int32_t next = j0 + kWaves * TK;
            const bool edge = j0 < low_max || j0 + TK - 1 > pos_min || j0 + TK - 1 > s1;
            F4 st[MB][2 * NB];
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
                for (int t = 0; t < 2 * NB; ++t) {
                    st[mb][t] = F4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        st[mb][t] = Frag<T>::mma(k_frag(x, t, k),
                                                 MB == 1 ? q1[k] : qf[(mb * KS + k) * kWave + lane],
                                                 st[mb][t]);
                }
            }
            pg = pn;
            if (next <= s1) {
                load_k(x, kc, pg.k, next, ends, g, h, lane);
                if (next + kWaves * TK <= s1)
                    pn = pages_of(g, b, next + kWaves * TK, ends, lane, bad);
            }
            U4 pf[MB][NB];
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                if (edge) {
#pragma unroll
                    for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int32_t j = j0 + grp * (8 * NB) + t * 4 + r;
                            if (j > pos[mb] || j < low[mb] || j > s1)
                                st[mb][t][r] = -INFINITY;
                        }
                }
                float mx = fmaxf(fmaxf(st[mb][0][0], st[mb][0][1]),
                                 fmaxf(st[mb][0][2], st[mb][0][3]));
#pragma unroll
                for (int t = 1; t < 2 * NB; ++t)
                    mx = fmaxf(mx, fmaxf(fmaxf(st[mb][t][0], st[mb][t][1]),
                                         fmaxf(st[mb][t][2], st[mb][t][3])));
                mx *= c;
                if (__any(mx > m[mb] + kSlack)) {
                    mx = fmaxf(mx, __shfl_xor(mx, 16));
                    mx = fmaxf(mx, __shfl_xor(mx, 32));
                    const float mn = fmaxf(m[mb], mx);
                    const float f = __builtin_amdgcn_exp2f(m[mb] - mn);
                    m[mb] = mn;
                    l[mb] *= f;
#pragma unroll
                    for (int i = 0; i < DB; ++i)
                        o[mb][i] *= f;
                }
                const float shift = kLift - m[mb];
#pragma unroll
                for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float p = __builtin_amdgcn_exp2f(fmaf(st[mb][t][r], c, shift));
                        st[mb][t][r] = p;
                        l[mb] += p;
                    }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    pf[mb][nb] = U4{pack2<T>(st[mb][2 * nb][0], st[mb][2 * nb][1]),
                                    pack2<T>(st[mb][2 * nb][2], st[mb][2 * nb][3]),
                                    pack2<T>(st[mb][2 * nb + 1][0], st[mb][2 * nb + 1][1]),
                                    pack2<T>(st[mb][2 * nb + 1][2], st[mb][2 * nb + 1][3])};
            }
            if (edge)
                hide(x, o, st, pos, low, vc, b, j0, s1, g, h, lane);
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const U4 vf = v_frag(x, i, nb);
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
                        o[mb][i] = Frag<T>::mma(vf, pf[mb][nb], o[mb][i]);
                }
            if (next <= s1)
                load_v(x, vc, pg.v, next, ends, g, h, lane);
        }

        // join the wavefronts: common maxima, then each sums a share of the dims
        const float vs = g.v_scale ? g.v_scale[h] : 1.0f;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            l[mb] += __shfl_xor(l[mb], 16);
            l[mb] += __shfl_xor(l[mb], 32);
            if (grp == 0)
                lds_ml[wave * M + mb * 16 + col] = float2{m[mb], l[mb]};
        }
        // (also: every wavefront is done with qf)
        const int64_t at = (((int64_t)b * g.kv_heads + h) * sp.splits + split) * (sp.m_tiles * M);
        if (__syncthreads_or(bad)) {
            if (threadIdx.x == 0)
                atomicOr(g.err, (uint32_t)kErrPage);
            if (whole) {
                fill_nan(out, lse, g, h, G, m0, m1);
                return;
            }
            for (int32_t r = m0 + threadIdx.x; r < m1; r += kWaves * kWave)
                sp.ml[at + r] = float2{0.0f, NAN};
            for (int32_t i = threadIdx.x; i < (m1 - m0) * D; i += kWaves * kWave)
                sp.o[(at + m0) * D + i] = NAN;
            return;
        }
        F4 *acc = (F4 *)lds;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            float top = -FLT_MAX, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                top = fmaxf(top, lds_ml[w * M + mb * 16 + col].x);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float2 y = lds_ml[w * M + mb * 16 + col];
                sum += y.y * __builtin_amdgcn_exp2f(y.x - top);
            }
            const float f = __builtin_amdgcn_exp2f(m[mb] - top) * vs;
            if (mb > 0)
                __syncthreads();
#pragma unroll
            for (int i = 0; i < DB; ++i)
                acc[(wave * DB + i) * kWave + lane] = o[mb][i] * f;
            __syncthreads();
            const int32_t row = m0 + mb * 16 + col;
            const bool live = row < m1;
            const int32_t t = row / G, hd = h * G + row - t * G;
            const float inv = whole ? 1.0f / sum : 1.0f;
            for (int i = wave; i < DB; i += kWaves) {
                F4 y = acc[i * kWave + lane];
#pragma unroll
                for (int w = 1; w < kWaves; ++w)
                    y += acc[(w * DB + i) * kWave + lane];
                if (!live)
                    continue;
                if (whole) {
                    y *= inv;
                    *(U2 *)(out + ((int64_t)t * g.q_heads + hd) * D + i * 16 + grp * 4) =
                        U2{pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3])};
                } else {
                    *(F4 *)(sp.o + (at + row) * D + i * 16 + grp * 4) = y;
                }
            }
            if (live && wave == 0 && grp == 0) {
                if (whole) {
                    if (lse)
                        lse[(int64_t)t * g.q_heads + hd] = (top - kLift) * kLn2 + __logf(sum);
                } else {
                    sp.ml[at + row] = float2{top, sum};
                }
            }
        }
    }

    // NaN in rows [m0, m0 + M) below `end` of a request.
    static __device__ void fill_nan(T *out, float *lse, const BlockArgs &g, int32_t h, int32_t G,
                                    int32_t m0, int32_t end)
    {
        const int32_t m1 = m0 + M < end ? m0 + M : end;
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
    static __device__ void hide(Tile &x, F4 (&o)[MB][DB], const F4 (&st)[MB][2 * NB],
                                const int32_t (&pos)[MB], const int32_t (&low)[MB], const C *vc,
                                int32_t b, int32_t j0, int32_t s1, const BlockArgs &g, int32_t h,
                                int lane)
    {
        const int grp = lane >> 4;
        const int32_t left = s1 - (j0 + grp * (8 * NB));  // slots 0..left are in the span
        constexpr int kPer = kByte ? 4 : 2;               // cells of a 32-bit word
        constexpr uint32_t kBits = kByte ? 0xffu : 0xffffu;
        // NaN (and infinity): all ones in the exponent (8-bit: in all but the sign)
        constexpr uint32_t kExp = kByte ? 0x7fu : (sizeof(typename Frag<T>::V2) == 4 &&
                                                           __is_same(T, __bf16)
                                                       ? 0x7f80u
                                                       : 0x7c00u);
        uint32_t odd = 0;  // slots with such a cell
#pragma unroll
        for (int e = 0; e < 8 * NB; ++e) {
            const uint32_t mask = kBits << (e % kPer * (32 / kPer));
            bool any = false;
#pragma unroll
            for (int i = 0; i < DB; ++i) {
                const uint32_t w = x.v[i][e / kPer] >> (e % kPer * (32 / kPer));
                any |= (w & kExp) == kExp;
            }
            any &= e <= left;
            const uint64_t vote = __ballot(any);
            if ((vote >> (grp * 16)) & 0xffffu)
                odd |= 1u << e;
            if (e > left || ((odd >> e) & 1)) {
#pragma unroll
                for (int i = 0; i < DB; ++i)
                    x.v[i][e / kPer] &= ~mask;
            }
        }
        if (!__any(odd != 0))
            return;
        const int32_t tokens = 1 << g.page_shift;
        for (int from = 0; from < 4; ++from) {
#pragma unroll
            for (int e = 0; e < 8 * NB; ++e) {
                if (!((__shfl(odd, from * 16) >> e) & 1))
                    continue;
                const int32_t j = j0 + from * (8 * NB) + e;
                const int32_t page = page_of(g, b, j), id = page < 0 ? 0 : page;
                const C *p = vc + (((int64_t)id * g.kv_heads + h) * D + grp * 4) * tokens +
                             (j & (tokens - 1));
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    const float w = to_f32((T)__shfl(st[mb][e / 4][e % 4], from * 16 + (lane & 15)));
                    if (j <= pos[mb] && j >= low[mb]) {
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

template <typename T, typename C, int D, int MB>
__global__ __launch_bounds__(kWaves *kWave) void attend_kernel(AttendArgs a, Split sp)
{
    __shared__ __attribute__((aligned(16))) char lds[Kernel<T, C, D, MB>::kLds];
    __shared__ float2 lds_ml[kWaves * 16 * MB];
    Kernel<T, C, D, MB>::run(a, sp, lds, lds_ml);
}

// Joins the spans of a row: one wavefront per (request, row, query head).
template <typename T, int D, int TK, int M>
__global__ __launch_bounds__(kWave) void join_kernel(AttendArgs a, Split sp)
{
    const BlockArgs &g = a.blk;
    const int32_t lane = threadIdx.x, hd = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    int32_t length;
    uint32_t err;
    const int32_t n = block_rows(g, b, length, err);
    if (t >= n)
        return;
    const int32_t G = g.q_heads / g.kv_heads, h = hd / G;
    const int32_t row = t * G + hd - h * G, m0 = row / M * M;
    const int32_t m1 = m0 + M < n * G ? m0 + M : n * G;
    const Sight s = sight_of<TK>(a, length, m0 / G, (m1 - 1) / G);
    const int32_t spans = (s.hi - s.start) / sp.span + 1;
    if (spans == 1)
        return;
    const int64_t rows = (int64_t)sp.m_tiles * M;
    const int64_t at = ((int64_t)b * g.kv_heads + h) * sp.splits * rows + row;
    float top = -FLT_MAX;
    for (int32_t i = lane; i < spans; i += kWave)
        top = fmaxf(top, sp.ml[at + i * rows].x);
    for (int i = kWave / 2; i; i >>= 1)
        top = fmaxf(top, __shfl_xor(top, i));
    float sum = 0.0f, y[(D + kWave - 1) / kWave] = {};
    for (int32_t i = 0; i < spans; ++i) {
        const float2 v = sp.ml[at + i * rows];
        const float f = __builtin_amdgcn_exp2f(v.x - top);
        sum += v.y * f;
#pragma unroll
        for (int k = 0; k < (D + kWave - 1) / kWave; ++k)
            if (k * kWave + lane < D)
                y[k] += f * sp.o[(at + i * rows) * D + k * kWave + lane];
    }
    const int64_t r = ((int64_t)b * g.rows + t) * g.q_heads + hd;
#pragma unroll
    for (int k = 0; k < (D + kWave - 1) / kWave; ++k)
        if (k * kWave + lane < D)
            ((T *)a.out)[r * D + k * kWave + lane] = from_f32<T>(y[k] / sum);
    if (a.out_lse && lane == 0)
        a.out_lse[r] = (top - kLift) * kLn2 + __logf(sum);
}

// Query-row blocks of a workgroup: 1, 2 or 4, at most 512 / D (registers).
int row_blocks(int32_t rows, int32_t group, int32_t dim)
{
    const int64_t m = (int64_t)rows * group;
    int mb = m <= 16 ? 1 : (m <= 32 ? 2 : 4);
    while (mb * dim > 512)
        mb /= 2;
    return mb;
}

// Positions of a span: enough workgroups that ragged requests even out, but
// at least 32 positions for each query row, so that the partial results
// (8 bytes a dim written and read, against 4 of cache) stay a small share.
constexpr int64_t kTargetGroups = 4096;
constexpr int32_t kMinSpan = 256;

int64_t span_of(int64_t positions, int64_t groups, int m, int tile)
{
    int64_t span = (positions * groups + kTargetGroups - 1) / kTargetGroups;
    if (span < kMinSpan)
        span = kMinSpan;
    if (span < 32 * m)
        span = 32 * m;
    span = (span + kWaves * tile - 1) / (kWaves * tile) * (kWaves * tile);
    return span;
}

template <typename T, typename C, int D, int MB>
hipError_t launch_full(const AttendArgs &a, hipStream_t s)
{
    typedef Kernel<T, C, D, MB> K;
    const BlockArgs &g = a.blk;
    const int64_t m = (int64_t)g.rows * (g.q_heads / g.kv_heads);
    Split sp;
    sp.m_tiles = (int32_t)((m + K::M - 1) / K::M);
    const int64_t sight = a.window && (int64_t)a.window + g.rows - 1 < g.max_len
                              ? (int64_t)a.window + g.rows - 1 + K::TK
                              : g.max_len;
    const int64_t groups = (int64_t)g.batch * g.kv_heads * sp.m_tiles;
    // the workspace holds the partial results of so many spans
    const int64_t room = a.ws_rows / (groups * K::M), tile = kWaves * K::TK;
    int64_t span = span_of(sight, groups, K::M < m ? K::M : (int)m, K::TK);
    const int64_t fit = room < 2 ? sight : (sight + room - 1) / room;
    if (span < fit)
        span = (fit + tile - 1) / tile * tile;
    const int64_t splits = (sight + span - 1) / span;
    sp.span = span < 0x7fffffffLL ? (int32_t)span : 0x7fffffff;
    sp.splits = (int32_t)splits;
    sp.o = a.ws;
    sp.ml = (float2 *)(a.ws + a.ws_rows * D);
    const int64_t chunks = ((int64_t)g.batch * g.kv_heads * splits + 7) / 8 * 8;
    if (chunks * sp.m_tiles > 0x7fffffffLL)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((attend_kernel<T, C, D, MB>), dim3((uint32_t)(chunks * sp.m_tiles)),
                       dim3(kWaves * kWave), 0, s, a, sp);
    if (splits > 1)
        hipLaunchKernelGGL((join_kernel<T, D, K::TK, K::M>), dim3(g.q_heads, g.rows, g.batch),
                           dim3(kWave), 0, s, a, sp);
    return hipGetLastError();
}

template <typename T, typename C, int D>
hipError_t launch_dim(const AttendArgs &a, hipStream_t s)
{
    const int mb = row_blocks(a.blk.rows, a.blk.q_heads / a.blk.kv_heads, D);
    if (mb == 1)
        return launch_full<T, C, D, 1>(a, s);
    if constexpr (D <= 128)
        if (mb == 4)
            return launch_full<T, C, D, 4>(a, s);
    return launch_full<T, C, D, 2>(a, s);
}

template <typename T, typename C>
hipError_t launch_typed(const AttendArgs &a, hipStream_t s)
{
    switch (a.blk.head_dim) {
    case 64: return launch_dim<T, C, 64>(a, s);
    case 96: return launch_dim<T, C, 96>(a, s);
    case 128: return launch_dim<T, C, 128>(a, s);
    case 192: return launch_dim<T, C, 192>(a, s);
    default: return launch_dim<T, C, 256>(a, s);
    }
}

}  // namespace

// Enough for kTargetGroups workgroups of the widest tile (64 rows), or for
// every span of the shortest kind that the context's calls can have.
int64_t attend_rows(const pld_target_params &p)
{
    const int64_t group = p.q_heads / p.kv_heads;
    const int64_t rows = (p.max_rows * group + 63) / 64 * 64 * p.max_batch * p.kv_heads;
    const int64_t spans = (p.max_len + kMinSpan - 1) / kMinSpan;
    const int64_t most = 64 * kTargetGroups;
    return spans >= (most + rows - 1) / rows ? most : rows * spans;
}

hipError_t launch_attend(const AttendArgs &a, hipStream_t s)
{
    const bool wide = a.blk.cache_dtype != PLD_E4M3;
    if (a.blk.dtype == PLD_BF16)
        return wide ? launch_typed<__bf16, __bf16>(a, s) : launch_typed<__bf16, E4m3>(a, s);
    return wide ? launch_typed<_Float16, _Float16>(a, s) : launch_typed<_Float16, E4m3>(a, s);
}

}  // namespace pld
