// Attention of a tree's many rows over the paged cache, for gfx950 (MI355X):
// more than 32 query rows a kv head.
//
// Mathematics as in pld_attend_device.h, in 32x32x16 matrix instructions: a
// wavefront holds 32 query rows, a lane half of the positions of one of them.
// With so many rows the matrix and vector units bound it, not the cache: a score
// costs 1/128 of a product's operands twice and one exponential. What was done
// about it, and what it gave for 16 requests of 131,072 positions, 2 kv heads of 128
// and 512 query rows (1.10 TFLOP; the 16x16 kernel of pld_attend_device.h: 1,602 us):
//  - tiles of 64 positions, one barrier each; a tile goes into LDS row by row as it
//    lies in memory (whole lines), by direct loads whose addresses are a scalar's
//    page and a lane's constants: 1,509;
//  - the 16-byte chunks of a row exchanged so that 16 neighbouring lanes read all
//    of the LDS's banks (half of its cycles were conflicts), and operands read two
//    groups ahead of the product that takes them: 1,367;
//  - the weights of one half of a tile worked out between the other half's
//    products, masks kept to tiles where sights end: 1,350; a wavefront at its
//    products before one at its weights: 1,300 to 1,335, 824 to 846 TFLOP/s, three
//    fifths of what a large product reaches here.
// Its fetches take a quarter of that (1,021 us with the first tiles read over and
// over); the rest is the two units taking turns. The cache is read from HBM once:
// 2.17 GB counted, the other three workgroups of a span find it in L2.
// Tried and not kept: K fetched two tiles ahead, V one and a half (1,360); 8
// wavefronts that share a tile (1,424: they wait for each other); 64 query rows a
// wavefront, one a SIMD (2,540: its registers spill).
//
// 8-bit cells go through registers, where each is widened once for the workgroup:
// 64 ragged requests of 8,192 to 65,536 positions, 4 kv heads of 128, up to 96 query
// rows: 1,491 us when every wavefront widened for itself, 752 to 863 now, 2.8 to 3.2
// TB/s; a span's start, its widening and its products follow each other there.
#pragma once

#include "pld_attend_device.h"

namespace pld {

namespace {

typedef float F16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ F16 mma32(U4 a, U4 b, F16 c, __bf16)
{
    typedef Frag<__bf16>::V8 V8;
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(V8, a),
                                                   __builtin_bit_cast(V8, b), c, 0, 0, 0);
}
__device__ __forceinline__ F16 mma32(U4 a, U4 b, F16 c, _Float16)
{
    typedef Frag<_Float16>::V8 V8;
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(V8, a),
                                                  __builtin_bit_cast(V8, b), c, 0, 0, 0);
}

template <typename T, typename C, int D>
struct Tall : Tiles<T, C, D, 1, true> {
    typedef Tiles<T, C, D, 1, true> S;
    static_assert(D == 64 || D == 128, "rows that are whole LDS lines");
    static constexpr bool kByte = sizeof(C) == 1;
    static constexpr int TK = 64;                  // positions of a tile
    static constexpr int kGrain = TK;
    static constexpr int64_t kSpanBytes = 1 << 20;
    static constexpr int M = 32 * kWaves;
    static constexpr int KS = D / 16;              // steps of K Q^T
    static constexpr int DB = D / 32;              // blocks of 32 dims
    static constexpr int kRow = D * 2;             // bytes of a K row in LDS
    static constexpr int kKeys = TK * kRow;        // bytes of a tile's K, and of its V
    static constexpr int kStage = 2 * kKeys;
    // (M0 holds 16 bits of an LDS address)
    static constexpr int kStages = kByte ? 2 : 65536 / kStage;
    static constexpr int kLoads = kKeys / (kWaves * 1024);  // of K, of V: a wavefront, a tile
    static constexpr int kUnits = D / 64;          // 8-bit words of K, of V: a thread, a tile
    static constexpr int kBranches = kStages * kStage;
    static constexpr int kOdd = kBranches + Branches::kLds;
    static constexpr int kLds = kOdd + 16;
    static constexpr int kGroups = 2 * KS / 4;     // of K's operands
    typedef typename S::Pages Pages;

    // A chunk of 16 bytes, c of K's row r, stands in place c ^ k_turn(r) of the
    // row, c of V's row of dim d in c ^ v_turn(d): the chunks c of 16 rows side
    // by side then lie in 16 different places of the 256 bytes that the LDS
    // reads at once. (V's rows are 128 bytes. Bit 3 of the dim, in which two
    // loads differ, turns neighbouring chunks: they are in one page.)
    static __device__ __forceinline__ int k_turn(int r)
    {
        return D == 128 ? r & 15 : r >> 1 & 7;
    }
    static __device__ __forceinline__ int v_turn(int d) { return (d >> 3 & 1) | (d & 6); }

    // What brings tiles: the caches' parts of this kv head, and a lane's
    // constants.
    struct Bring {
        const char *k, *v;
        int64_t page_bytes;
        int32_t tokens;
        uint32_t k_off[4];   // of each load: bytes behind the wavefront's 16 rows
        uint32_t v_off;      // bytes of its dim's row behind the page
        int32_t v_at;        // its positions behind the tile's start
        int32_t v_odd;       // bytes that odd loads lie further
    };
    static __device__ __forceinline__ Bring bring_of(const AttendArgs &a, int32_t h, int lane,
                                                     int wave)
    {
        Bring x;
        const BlockArgs &g = a.blk;
        x.tokens = 1 << g.page_shift;
        const int64_t head = (int64_t)x.tokens * D * sizeof(C);
        x.page_bytes = g.kv_heads * head;
        x.k = (const char *)a.k_cache + h * head;
        x.v = (const char *)a.v_cache + h * head;
        if constexpr (kByte) {
            const int tid = wave * kWave + lane;
            for (int n = 0; n < 4; ++n)
                x.k_off[n] = tid / (D / 16) % 16 * D + tid % (D / 16) * 16;
            x.v_off = tid / 4 * x.tokens;
            x.v_at = tid % 4 * 16;
            x.v_odd = 0;
        } else {
            constexpr int kChunks = kRow / 16;
            const int r = lane / kChunks;
            for (int n = 0; n < 4; ++n)
                x.k_off[n] = r * kRow +
                             ((lane % kChunks) ^ k_turn(n * (kWave / kChunks) + r)) * 16;
            const int chunk = (lane % 8) ^ v_turn(lane / 8);
            x.v_off = (wave * (D / kWaves) + lane / 8) * x.tokens * 2;
            x.v_at = chunk * 8;
            x.v_odd = chunk % 2 ? -16 : 16;
        }
        return x;
    }
    static __device__ __forceinline__ int32_t page_for(const Pages &p, int quarter)
    {
        const int32_t x = p.x, y = p.y, z = p.z, w = p.w;
        const int32_t lo = (quarter & 1) ? y : x, hi = (quarter & 1) ? w : z;
        return (quarter & 2) ? hi : lo;
    }
    // Where this lane's V of the tile at j0 starts.
    static __device__ __forceinline__ const char *v_from(const Bring &x, const Pages &p,
                                                         int32_t j0)
    {
        return x.v + page_for(p, x.v_at >> 4) * x.page_bytes +
               (x.v_off + ((j0 + x.v_at) & (x.tokens - 1)) * (uint32_t)sizeof(C));
    }

    // 16-bit cells: a tile's direct loads into the stage at LDS address `to`. A
    // load's offset goes for both addresses.
    static __device__ __forceinline__ void fetch(const Bring &x, const Pages &p, int32_t j0,
                                                 uint32_t to, int wave)
    {
        const char *k = x.k + page_for(p, wave) * x.page_bytes +
                        (int64_t)((j0 + wave * 16) & (x.tokens - 1)) * kRow;
        const uint32_t k_to = __builtin_amdgcn_readfirstlane(to + wave * 16 * kRow);
        const uint32_t v_to =
            __builtin_amdgcn_readfirstlane(to + kKeys + wave * (D / kWaves) * (TK * 2));
        uint32_t m0;
        // (M0, the LDS address, is the compiler's: put back; a load may not
        // follow its write at once)
        if constexpr (kLoads == 4)
            asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %6\n\ts_nop 0\n\t"
                         "global_load_lds_dwordx4 %1, %5\n\t"
                         "global_load_lds_dwordx4 %2, %5 offset:1*1024\n\t"
                         "global_load_lds_dwordx4 %3, %5 offset:2*1024\n\t"
                         "global_load_lds_dwordx4 %4, %5 offset:3*1024\n\ts_mov_b32 m0, %0"
                         : "=&s"(m0)
                         : "v"(x.k_off[0]), "v"(x.k_off[1]), "v"(x.k_off[2]), "v"(x.k_off[3]),
                           "s"(k), "s"(k_to)
                         : "memory");
        else
            asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %4\n\ts_nop 0\n\t"
                         "global_load_lds_dwordx4 %1, %3\n\t"
                         "global_load_lds_dwordx4 %2, %3 offset:1*1024\n\ts_mov_b32 m0, %0"
                         : "=&s"(m0)
                         : "v"(x.k_off[0]), "v"(x.k_off[1]), "s"(k), "s"(k_to)
                         : "memory");
        const uint32_t step = 8 * x.tokens * 2;
        if (x.tokens >= TK) {
            // one page a tile: a scalar's address and a lane's constants
            const char *v = x.v + p.x * x.page_bytes + (int64_t)(j0 & (x.tokens - 1)) * 2;
#pragma unroll
            for (int n = 0; n < kLoads; ++n)
                asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\t"
                             "global_load_lds_dwordx4 %1, %2\n\ts_mov_b32 m0, %0"
                             : "=&s"(m0)
                             : "v"(x.v_off + x.v_at * 2 + (n & 1) * x.v_odd), "s"(v + n * step),
                               "s"(v_to + n * 1024)
                             : "memory");
            return;
        }
        const char *v = v_from(x, p, j0);
#pragma unroll
        for (int n = 0; n < kLoads; ++n)
            asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\t"
                         "global_load_lds_dwordx4 %1, off\n\ts_mov_b32 m0, %0"
                         : "=&s"(m0)
                         : "v"(v + (int32_t)(n * step + (n & 1) * x.v_odd)), "s"(v_to + n * 1024)
                         : "memory");
    }

    // 8-bit cells: a tile's words of this thread, and their way into a stage.
    struct Words {
        U4 k[kUnits], v[kUnits];
    };
    static __device__ __forceinline__ void load(Words &y, const Bring &x, const Pages &p,
                                                int32_t j0, int wave)
    {
#pragma unroll
        for (int n = 0; n < kUnits; ++n) {
            const int rows = D == 128 ? wave / 2 + n * 2 : wave;  // which 16
            y.k[n] = *(const U4 *)(x.k + page_for(p, rows) * x.page_bytes +
                                   (int64_t)((j0 + rows * 16) & (x.tokens - 1)) * D + x.k_off[0]);
        }
        const char *v = v_from(x, p, j0);
#pragma unroll
        for (int n = 0; n < kUnits; ++n)
            y.v[n] = *(const U4 *)(v + n * 64 * x.tokens);
    }
    static __device__ __forceinline__ void put(char *row, int chunk, int turn, U4 w)
    {
        *(U4 *)(row + (chunk ^ turn) * 16) = widen8<T>(w[0], w[1]);
        *(U4 *)(row + ((chunk + 1) ^ turn) * 16) = widen8<T>(w[2], w[3]);
    }
    static __device__ __forceinline__ void spread(const Words &y, char *stage, int tid)
    {
#pragma unroll
        for (int n = 0; n < kUnits; ++n) {
            const int r = tid / (D / 16) + n * 32;
            put(stage + r * kRow, tid % (D / 16) * 2, k_turn(r & 15), y.k[n]);
            const int d = tid / 4 + n * 64;
            put(stage + kKeys + d * (TK * 2), tid % 4 * 2, v_turn(d), y.v[n]);
        }
    }

    // A tile where a sight ends: V of positions past the span's end becomes
    // zero, and so does each element that is an infinity or a NaN (0 times it
    // would be NaN in the rows that do not see it); returns the positions that
    // hold such elements, which the rows that see them then add. The other
    // elements of such a position stay, for the products. Barriers stand before
    // and behind it.
    static __device__ __forceinline__ uint64_t clean(char *stage, uint32_t *odd, int32_t last)
    {
        constexpr uint32_t kExp = __is_same(T, __bf16) ? 0x7f80u : 0x7c00u;
        uint64_t mine = 0;
        for (int u = threadIdx.x; u < D * 8; u += kWaves * kWave) {
            U4 *const w = (U4 *)(stage + kKeys) + u;
            const int at = ((u & 7) ^ v_turn(u >> 3)) * 8;
            U4 y = *w;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t mask = 0xffffu << (e % 2 * 16);
                const bool past = at + e > last;
                const bool wild = ((y[e / 2] >> (e % 2 * 16)) & kExp) == kExp;
                if (past || wild)
                    y[e / 2] &= ~mask;
                if (wild && !past)
                    mine |= 1ull << (at + e);
            }
            *w = y;
        }
        if (!__syncthreads_or(mine != 0))
            return 0;
        if (threadIdx.x < 2)
            odd[threadIdx.x] = 0;
        __syncthreads();
        if ((uint32_t)mine)
            atomicOr(odd, (uint32_t)mine);
        if ((uint32_t)(mine >> 32))
            atomicOr(odd + 1, (uint32_t)(mine >> 32));
        __syncthreads();
        const uint64_t all = (uint64_t)odd[1] << 32 | odd[0];
        __syncthreads();
        return all;
    }

    // The order of a stretch of code: GROUPS times N products, each with its
    // share of 56 vector operations behind it, then the reads of a group.
    template <int GROUPS, int N> static __device__ __forceinline__ void interleave()
    {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 56 / (GROUPS * N), 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
        }
    }

    // HALVES: rows for two wavefronts only (a ragged tree): two take the first 32
    // positions of a tile and two the others, and join at the end. (A function of
    // its own: with both in one the registers spill, 3,110 us against 1,150.)
    template <bool HALVES>
    static __device__ __forceinline__ void run(const AttendArgs &a, const Split &sp, char *lds,
                                               const Work &w)
    {
        const BlockArgs &g = a.blk;
        const int tid = threadIdx.x, lane = tid & (kWave - 1);
        const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
        const int grp = lane >> 5, col = lane & 31;
        // (pages are looked up for 16 positions each)
        const typename S::Ends ends{(w.lo > w.s0 ? w.lo : w.s0) / 16 * 16, w.s1 / 16 * 16};
        const int32_t root = w.length - 1;
        const bool branchy = w.s1 > root || a.window;
        int32_t up = 0;
        bool stray = false, bad = false;
        if (branchy)
            up = parent_of(a.parent, g, w.b, tid, stray);
        const auto pages_at = [&](int32_t j0) {
            Pages p;
            p.x = S::page_at(g, w.b, j0, ends, bad);
            p.y = p.z = p.w = p.x;
            if (g.page_shift >= 6)
                return p;
            p.y = S::page_at(g, w.b, j0 + 16, ends, bad);
            p.z = S::page_at(g, w.b, j0 + 32, ends, bad);
            p.w = S::page_at(g, w.b, j0 + 48, ends, bad);
            return p;
        };

        const Bring x = bring_of(a, w.h, lane, wave);
        const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
        const int32_t tiles = (w.s1 - w.s0) / TK + 1;
        Words next;
        Pages pn = pages_at(w.s0);
        if constexpr (kByte) {
            load(next, x, pn, w.s0, wave);
            spread(next, lds, tid);
            pn = pages_at(w.s0 + TK);
            if (tiles > 1)
                load(next, x, pn, w.s0 + TK, wave);
            pn = pages_at(w.s0 + 2 * TK);
        } else {
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) {
                if (i < tiles)
                    fetch(x, pn, w.s0 + i * TK, ring + i * kStage, wave);
                pn = pages_at(w.s0 + (i + 1) * TK);
            }
        }

        const char *const branches = lds + kBranches;
        if (branchy) {
            if (__syncthreads_or(stray)) {
                // (its LDS is another workgroup's once this one ends)
                asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
                give_up<Tall, T, D>(a, sp, w, kErrBlock);
                return;
            }
            Branches::build(lds + kBranches, up, g.draft_len[w.b] + 1, a.window);
        }

        const int mine = HALVES ? wave >> 1 : 0;

        // this lane's query row
        const float ks = g.k_scale ? g.k_scale[w.h] : 1.0f;
        const float c0 = a.scale * ks * kLog2e;
        const float c = factor(c0);
        const uint32_t flip = c0 < 0.0f ? 0x80008000u : 0u;
        const int32_t row = w.m0 + (HALVES ? wave & 1 : wave) * 32 + col;
        int32_t node, low;
        {
            const int32_t in = row < w.m1 ? row : w.m1 - 1;
            S::sight_of_row(a, in / w.G, root, branches, node, low);
        }
        U4 q[KS];
        {
            const int32_t t = row / w.G;
            const T *from = (const T *)a.q + ((int64_t)w.b * g.rows + t) * a.q_stride +
                            (int64_t)(w.h * w.G + row - t * w.G) * D + grp * 8;
#pragma unroll
            for (int s = 0; s < KS; ++s)
                q[s] = row < w.m1 ? *(const U4 *)(from + s * 16) ^ flip : U4{0u, 0u, 0u, 0u};
        }
        const int32_t end = w.length - 1 + (w.m1 - 1) / w.G;
        const int32_t all_from = a.window && end >= a.window ? end - a.window + 1 : 0;

        // where this lane's operands of a stage stand: K's row i is position
        // i with its bits 2 and 3 exchanged, so that the scores of a lane are
        // eight positions side by side, twice: the operand that V takes
        const int pos = (col & 0x13) | (col >> 1 & 4) | (col << 1 & 8);
        uint32_t k_at[KS], v_at[4];
#pragma unroll
        for (int n = 0; n < KS; ++n)
            k_at[n] = pos * kRow + ((2 * n + grp) ^ k_turn(pos & 15)) * 16;
#pragma unroll
        for (int n = 0; n < 4; ++n)
            v_at[n] = kKeys + col * (TK * 2) + ((2 * n + grp) ^ v_turn(col)) * 16;

        float m = -FLT_MAX, l = 0.0f, fall = 1.0f;
        F16 o[DB];
#pragma unroll
        for (int i = 0; i < DB; ++i)
            o[i] = F16{};
        int slot = 0;
        for (int32_t i = 0; i < tiles; ++i) {
            const int32_t j0 = w.s0 + i * TK;
            char *const stage = lds + slot * kStage;
            if constexpr (kByte) {
                // (also: every wavefront is done with the other stage)
                __syncthreads();
            } else {
                // this wavefront's loads of tile i are done; the barrier stands
                // for the others', and for their reads of the slot that the
                // next fetch overwrites
                if (i + kStages - 2 < tiles)
                    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier"
                                 :
                                 : "n"(2 * kLoads * (kStages - 2))
                                 : "memory");
                else
                    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : : : "memory");
                const int32_t ahead = i + kStages - 1;
                if (ahead < tiles) {
                    fetch(x, pn, w.s0 + ahead * TK,
                          ring + (slot == 0 ? kStages - 1 : slot - 1) * kStage, wave);
                    pn = pages_at(w.s0 + (ahead + 1) * TK);
                }
            }
            slot = slot + 1 == kStages ? 0 : slot + 1;
            const bool edge = j0 < all_from || j0 + TK - 1 > root || j0 + TK - 1 > w.s1;
            uint64_t odd = 0;
            if (edge)
                odd = clean(stage, (uint32_t *)(lds + kOdd), w.s1 - j0);

            // (a wavefront before its products, which go one after the other, comes
            // before the one beside it that is at its weights)
            __builtin_amdgcn_s_setprio(1);
            // Two halves of 32 positions: the second's scores are on their way
            // while the first's probabilities are worked out, and the first's
            // products with V while the second's are. Operands are read two
            // groups ahead of the products that take them: 4 of K, DB of V.
            U4 f[2][4];
            const auto read = [&](int n) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (n < kGroups)
                        f[n & 1][k] = *(const U4 *)(stage + k_at[n * 4 % KS + k] +
                                                    n * 4 / KS * 32 * kRow);
                    else if (n < kGroups + 4 && k < DB)
                        f[n & 1][k] =
                            *(const U4 *)(stage + v_at[n - kGroups] + k * 32 * (TK * 2));
                }
            };
            F16 st[2] = {F16{}, F16{}};
            const auto scores = [&](int n) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    st[n * 4 / KS] = mma32(f[n & 1][k], q[n * 4 % KS + k], st[n * 4 / KS], T{});
                read(n + 2);
            };
            U4 pf[4];
            const auto sums = [&](int n) {
#pragma unroll
                for (int k = 0; k < DB; ++k)
                    o[k] = mma32(f[(n + kGroups) & 1][k], pf[n], o[k], T{});
                read(n + kGroups + 2);
            };
            const auto mask = [&](int pb, int32_t at) {
                // a bit for each of the lane's positions from j on
                const int32_t j = at + grp * 8, last = w.s1 - j, first = low - j;
                uint32_t seen = branchy ? Branches::bits(branches, node, j, root) : 0xffffffffu;
                seen &= last < 0 ? 0u : (last < 31 ? (2u << last) - 1u : 0xffffffffu);
                seen &= first <= 0 ? 0xffffffffu : (first < 32 ? 0xffffffffu << first : 0u);
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (!(seen & (1u << ((r >> 3) * 16 + (r & 7)))))
                        st[pb][r] = -INFINITY;
            };
            // raises the running maximum where a score is far above it: the
            // factor on what was summed with the old one, or 1
            const auto raise = [&](int pb) {
                float mx = fmaxf(st[pb][0], st[pb][1]);
#pragma unroll
                for (int r = 2; r < 16; ++r)
                    mx = fmaxf(mx, st[pb][r]);
                mx *= c;
                if (!__any(mx > m + kSlack))
                    return false;
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                const float mn = fmaxf(m, mx);
                fall = __builtin_amdgcn_exp2f(m - mn);
                m = mn;
                l *= fall;
                return true;
            };
            const auto weights = [&](int pb) {
                const float shift = kLift - m;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        y[e] = __builtin_amdgcn_exp2f(fmaf(st[pb][n * 8 + e], c, shift));
                        l += y[e];
                    }
                    pf[pb * 2 + n] = U4{pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]),
                                        pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7])};
                }
                // (they are worked out here, beside the products, and not where
                // they are used)
                asm volatile("" : : "v"(pf[pb * 2]), "v"(pf[pb * 2 + 1]), "v"(l));
            };
            const auto lower = [&] {
#pragma unroll
                for (int n = 0; n < DB; ++n)
                    o[n] *= fall;
            };
            if constexpr (HALVES) {
                const auto part = [&](int n) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (n < kGroups / 2)
                            f[n & 1][k] =
                                *(const U4 *)(stage + k_at[n * 4 + k] + mine * 32 * kRow);
                        else if (k < DB)
                            f[n & 1][k] = *(const U4 *)(stage +
                                                        (mine ? v_at[n - kGroups / 2 + 2]
                                                              : v_at[n - kGroups / 2]) +
                                                        k * 32 * (TK * 2));
                    }
                };
                part(0);
                part(1);
#pragma unroll
                for (int n = 0; n < kGroups / 2; ++n) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        st[0] = mma32(f[n & 1][k], q[n * 4 + k], st[0], T{});
                    __builtin_amdgcn_sched_barrier(0);
                    part(n + 2);
                }
                if (edge)
                    mask(0, j0 + mine * 32);
                if (raise(0))
                    lower();
                __builtin_amdgcn_s_setprio(0);
                weights(0);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int k = 0; k < DB; ++k)
                        o[k] = mma32(f[(n + kGroups / 2) & 1][k], pf[n], o[k], T{});
            } else {
                read(0);
                read(1);
#pragma unroll
                for (int n = 0; n < kGroups / 2; ++n)
                    scores(n);
                if (edge)
                    mask(0, j0);
                if (raise(0))
                    lower();
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = kGroups / 2; n < kGroups; ++n)
                    scores(n);
                weights(0);
                interleave<kGroups / 2, 4>();
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
                if (edge)
                    mask(1, j0 + 32);
                const bool raised = raise(1);
                __builtin_amdgcn_sched_barrier(0);
                sums(0);
                sums(1);
                weights(1);
                interleave<2, DB>();
                __builtin_amdgcn_sched_barrier(0);
                if (raised)
                    lower();
                sums(2);
                sums(3);
            }
            // elements that are not finite, for the rows that see them (no weight
            // changes what they make of a sum, so an older maximum's will do)
            if (HALVES)  // (those of its half)
                odd &= mine ? ~0ull << 32 : 0xffffffffull;
            for (; odd; odd &= odd - 1) {
                const int at = __builtin_ctzll(odd);
                const int32_t j = j0 + at, id = page_of(g, w.b, j);
                U4 four = pf[0];
#pragma unroll
                for (int n = 1; n < 4; ++n)
                    four = (HALVES ? at >> 4 & 1 : at >> 4) == n ? pf[n] : four;
                uint32_t two = four[0];
#pragma unroll
                for (int n = 1; n < 4; ++n)
                    two = (at >> 1 & 3) == n ? four[n] : two;
                two = __shfl(two, (at >> 3 & 1) * 32 + col) >> (at & 1) * 16;
                const float p = to_f32(__builtin_bit_cast(T, (uint16_t)two));
                const bool sees = !branchy || (Branches::bits(branches, node, j, root) & 1);
                if (j < low || !sees)
                    continue;
                const C *from = (const C *)(x.v + (id < 0 ? 0 : id) * x.page_bytes) +
                                grp * 4 * x.tokens + (j & (x.tokens - 1));
#pragma unroll
                for (int k = 0; k < DB; ++k)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float y =
                            to_f32(from[(k * 32 + (e >> 2) * 8 + (e & 3)) * x.tokens]);
                        if (!__builtin_isfinite(y))
                            o[k][e] += p * y;
                    }
            }
            if constexpr (kByte) {
                if (i + 1 < tiles) {
                    spread(next, lds + slot * kStage, tid);
                    if (i + 2 < tiles)
                        load(next, x, pn, j0 + 2 * TK, wave);
                    pn = pages_at(j0 + 3 * TK);
                }
            }
        }

        if (bad) {  // the same on every wavefront: they went through the same tiles
            give_up<Tall, T, D>(a, sp, w, kErrPage);
            return;
        }
        l += __shfl_xor(l, 32);
        if constexpr (HALVES) {
            // (the stages are done with)
            F4 *const other = (F4 *)lds + (wave & 1) * DB * 4 * kWave + lane;
            float2 *const other_ml = (float2 *)(lds + 2 * DB * 4 * kWave * 16) + (wave & 1) * kWave + lane;
            __syncthreads();
            if (mine) {
#pragma unroll
                for (int k = 0; k < DB; ++k)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        other[(k * 4 + u) * kWave] = F4{o[k][u * 4], o[k][u * 4 + 1],
                                                        o[k][u * 4 + 2], o[k][u * 4 + 3]};
                *other_ml = float2{m, l};
            }
            __syncthreads();
            if (mine)
                return;
            const float2 y = *other_ml;
            const float mn = fmaxf(m, y.x);
            const float f0 = __builtin_amdgcn_exp2f(m - mn), f1 = __builtin_amdgcn_exp2f(y.x - mn);
            m = mn;
            l = l * f0 + y.y * f1;
#pragma unroll
            for (int k = 0; k < DB; ++k)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[k][e] = o[k][e] * f0 + other[(k * 4 + e / 4) * kWave][e % 4] * f1;
        }
        if (row >= w.m1)
            return;
        const float vs = g.v_scale ? g.v_scale[w.h] : 1.0f;
        const float inv = 1.0f / l;
#pragma unroll
        for (int k = 0; k < DB; ++k)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const F4 y{o[k][u * 4] * vs, o[k][u * 4 + 1] * vs, o[k][u * 4 + 2] * vs,
                           o[k][u * 4 + 3] * vs};
                // (blocks of 16 dims, four lane groups of 4 in each)
                store<T, D>(a, sp, w, row, k * 2 + u / 2, (u & 1) * 2 + grp, y, inv);
            }
        if (grp == 0)
            store_ml(a, sp, w, row, m, l);
    }
};

template <typename T, typename C, int D>
__global__ __launch_bounds__(kWaves *kWave, 2) void attend_tall(AttendArgs a, Split sp)
{
    typedef Tall<T, C, D> K;
    __shared__ __attribute__((aligned(1024))) char lds[K::kLds];
    Work w;
    if (!work_of<K, T, K::M>(a, sp, w))
        return;
    if (w.m1 - w.m0 <= 64)
        K::template run<true>(a, sp, lds, w);
    else
        K::template run<false>(a, sp, lds, w);
}

}  // namespace

}  // namespace pld
