// Launches of the attention over the paged cache: the split of the positions and
// the rule that chooses the kernel.
#pragma once

#include "pld_attend_tall.h"

namespace pld {

namespace {

// Positions of a span. A workgroup streams about 14 KB a microsecond (two on
// each compute unit share what HBM gives) and takes some 10 us to start and
// to join, so a span should hold kSpanBytes of cache, as long as kEvenGroups
// workgroups can be had; never more than it takes for kMostGroups of them
// (ragged requests even out). A small batch is cut further to fill the chip,
// down to 32 positions a query row: the partial results are 8 bytes a dim,
// written and read, against 4 of cache. 16 x 262,144 positions, 128 rows:
// 985 us with 2 MiB, 918 with 4 MiB; 32 x 16,384, 64 rows: 294 us with 64
// positions a row, 236 with 32. (attend_tall, which its products bound, takes 1 MiB:
// the same within the spread from 512 KiB to 4 MiB with 16 bits a cell, and 1,155
// us against 1,182 with 2 MiB for 64 ragged requests of 8-bit cells.)
constexpr int64_t kFillGroups = 512;
constexpr int64_t kEvenGroups = 1024;
constexpr int64_t kMostGroups = 4096;
constexpr int32_t kMinSpan = 256;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Lays out a launch of kernel K and starts it, then the join.
template <typename K, typename T, int D, typename F>
hipError_t launch_split(const AttendArgs &a, F kernel, hipStream_t s)
{
    const BlockArgs &g = a.blk;
    const int64_t m = (int64_t)g.rows * (g.q_heads / g.kv_heads);
    Split sp;
    sp.m_tiles = (int32_t)((m + K::M - 1) / K::M);
    const int64_t sight = a.window && (int64_t)a.window + g.rows - 1 + K::TK < g.max_len
                              ? (int64_t)a.window + g.rows - 1 + K::TK
                              : g.max_len;
    const int64_t groups = (int64_t)g.batch * g.kv_heads * sp.m_tiles;
    const int64_t tile = K::kGrain, used = std::min<int64_t>(K::M, m);
    const int64_t total = sight * groups, bytes = 2 * D * K::kCellBytes;
    int64_t span = std::min<int64_t>(ceil_div(total, kFillGroups), 32 * used);
    span = std::max(span, std::min(ceil_div(total, kEvenGroups), K::kSpanBytes / bytes));
    span = std::max({span, ceil_div(total, kMostGroups), (int64_t)kMinSpan});
    // the workspace holds the partial results of so many spans
    const int64_t room = a.ws_rows / (groups * K::M);
    span = std::max(span, room < 2 ? sight : ceil_div(sight, room));
    span = ceil_div(span, tile) * tile;
    const int64_t splits = ceil_div(sight, span);
    sp.span = span < 0x7fffffffLL ? (int32_t)span : 0x7fffffff;
    sp.least = (int32_t)(ceil_div(std::max<int64_t>(kMinSpan, 32 * used), tile) * tile);
    sp.least = std::min(sp.least, sp.span);
    sp.splits = (int32_t)splits;
    sp.o = a.ws;
    sp.ml = (float2 *)(a.ws + a.ws_rows * D);
    const int64_t chunks = ceil_div((int64_t)g.batch * g.kv_heads * splits, 8) * 8;
    const int64_t joins = (int64_t)g.batch * g.rows * g.q_heads;
    if (!fits_grid(chunks * sp.m_tiles, kWaves * kWave) ||
        (splits > 1 && !fits_grid(joins, kWave)))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(chunks * sp.m_tiles)), dim3(kWaves * kWave), 0, s, a,
                       sp);
    if (splits > 1)
        hipLaunchKernelGGL((join_kernel<T, D, K::TK, K::M, K::kTree, K::kGrain>),
                           dim3((uint32_t)joins), dim3(kWave), 0, s, a, sp);
    return hipGetLastError();
}

// The kernel by the query rows of a kv head. Measured with 16-bit cells, 16
// requests of 65,536 positions and 2 kv heads, in us: narrow with 16 and 32 rows
// a workgroup, wide with 64 and 128. head_dim 128: 16 rows 202, 205, 207, 225; 17
// rows 277, 206, 208, 228; 32 rows 280, 212, 214, 234; 33 rows 416, 280, 217, 234;
// 64 rows 479, 285, 230, 248; 65 rows 650, 418, 320, 248. head_dim 256 (no narrow
// with 32): 16 rows 386, 546, 588; 17 rows 560, 548, 597; 64 rows 1,036, 573, 621;
// 65 rows 1,268, 944, 621. 8-bit cells take the same rule; there narrow with 32
// would hold out longer (head_dim 128, 64 rows: 144 against 168).
//
// Trees with more than 32 query rows take attend_tall where it has their head
// size. Measured, wide and tall, requests of 65,536 positions and 2 kv heads of
// 128: 44 rows, 16 requests, 8-bit cells 180 to 185 and 153 to 159, bf16 the same
// within the spread (223 to 228, 221 to 224); 64 rows 186 to 195 and 155 to 162,
// bf16 again the same (wide spreads over 233 to 272, tall over 231 to 233); 68 rows,
// bf16, 271 and 224; 128 rows 271 and 235, 8-bit 263 and 227; 2
// requests of 3,000 and 128 rows 27 and 25; 16 of 131,072 and 512 rows 1,602 and 1,300.
template <typename T, typename C, int D, bool TREE>
hipError_t launch_dim(const AttendArgs &a, hipStream_t s)
{
    const int64_t m = (int64_t)a.blk.rows * (a.blk.q_heads / a.blk.kv_heads);
    if (m <= 16)
        return launch_split<Narrow<T, C, D, 1, TREE>, T, D>(a, attend_narrow<T, C, D, 1, TREE>, s);
    if constexpr (D <= 128)
        if (m <= 32)
            return launch_split<Narrow<T, C, D, 2, TREE>, T, D>(a, attend_narrow<T, C, D, 2, TREE>,
                                                                s);
    if constexpr (TREE && (D == 64 || D == 128)) {
        return launch_split<Tall<T, C, D>, T, D>(a, attend_tall<T, C, D>, s);
    } else {
        if (m <= 64)
            return launch_split<Wide<T, C, D, 1, TREE>, T, D>(a, attend_wide<T, C, D, 1, TREE>, s);
        return launch_split<Wide<T, C, D, 2, TREE>, T, D>(a, attend_wide<T, C, D, 2, TREE>, s);
    }
}

template <typename T, typename C, bool TREE>
hipError_t launch_typed(const AttendArgs &a, hipStream_t s)
{
    switch (a.blk.head_dim) {
    case 64: return launch_dim<T, C, 64, TREE>(a, s);
    case 96: return launch_dim<T, C, 96, TREE>(a, s);
    case 128: return launch_dim<T, C, 128, TREE>(a, s);
    case 192: return launch_dim<T, C, 192, TREE>(a, s);
    default: return launch_dim<T, C, 256, TREE>(a, s);
    }
}

template <typename T, bool TREE>
hipError_t launch_blocks(const AttendArgs &a, hipStream_t s)
{
    return a.blk.cache_dtype == PLD_E4M3 ? launch_typed<T, E4m3, TREE>(a, s)
                                         : launch_typed<T, T, TREE>(a, s);
}

}  // namespace

}  // namespace pld
