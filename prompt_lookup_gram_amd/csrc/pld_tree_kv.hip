// The cache's writers of a tree's verification, for gfx950 (MI355X): norms,
// rotary positions by depth and the block's keys and values
// (pld_kv_append_tree), and the accepted path's cells moved side by side
// (pld_kv_keep).
//
// Mathematics: x -> w x / sqrt(mean x^2 + eps) over a head's dims, then the
// rotation of pld_kv.hip at the position of the row's depth. A head's sum of
// squares, its norm and its rotation are held in 32 bits, and it is rounded
// once.
//
// Bound by memory: every element is read and written once. A wavefront takes a
// row: it works out the row's depth and angles by itself and then streams the
// heads, 16 elements a lane (with the half layout a word and its partner in
// the pair), so that a head is a few lanes side by side, its sum a few
// exchanges, and no barrier stands anywhere. V is stored as in pld_kv.hip.
// 50,001 rows of 32 + 8 + 8 heads of 128 in bf16: 257 to 265 us back to back (265
// to 296 launch by launch under the trace), 4.6 to 4.8 TB/s read and written; a
// large copy reaches 4.5 to 5.0. 64 trees of up to 64 rows: 20 us for
// 51 MB; one tree of 16 rows 7.8, the chain of lengths, words, angles and stores.
// Two heads ahead instead of one: 23 and 277 us.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pld_kv_device.h"
#include "pld_tree_walk.h"

namespace pld {

namespace {

constexpr int kWave = 64;
constexpr int kWaves = kThreads / kWave;

template <int LANES>
__device__ __forceinline__ float lanes_sum(float x)
{
#pragma unroll
    for (int i = 1; i < LANES; i <<= 1)
        x += __shfl_xor(x, i);
    return x;
}

// 8 weights at any float's address.
struct __attribute__((packed, aligned(4))) Weights {
    float x[8];
};

// The factor of a head whose squares sum to `sum`.
__device__ __forceinline__ float norm_of(float sum, int32_t dim, float eps)
{
    return 1.0f / sqrtf(sum / (float)dim + eps);
}

// Words of 8 elements: q, k and v 16-byte aligned with strides of 8 elements,
// and rotated pairs that fill whole words. The first `turning` workgroups take
// kWaves rows each, the others store V. LANES lanes a head, 16 dims each: a
// power of two from head_dim / 16 on.
template <typename T, typename C, int LANES>
__global__ __launch_bounds__(kThreads) void tree_words(TreeAppendArgs ta, uint32_t turning,
                                                       uint32_t tiles)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const KvAppendArgs &a = ta.kv;
    const BlockArgs &g = a.blk;
    const int32_t dim = g.head_dim, tokens = 1 << g.page_shift, tid = threadIdx.x;
    const int lane = tid % kWave, wave = tid / kWave;
    WaveTree tree;
    if (blockIdx.x >= turning) {
        const uint32_t id = blockIdx.x - turning;
        // (every wavefront looks: they leave together)
        if (ta.parent && tree.load(ta.parent, g, id / (uint32_t)g.kv_heads / tiles, lane))
            return;
        store_values<T, C>(a, id, tiles, lds);
        return;
    }
    const uint32_t groups = (uint32_t)(g.rows + kWaves - 1) / kWaves;
    const int32_t b = blockIdx.x / groups;
    const int32_t t = __builtin_amdgcn_readfirstlane(blockIdx.x % groups * kWaves + wave);
    int32_t length;
    uint32_t err;
    const int32_t n = block_rows(g, b, length, err);
    if (t >= n) {
        if (err && t == 0 && lane == 0)
            atomicOr(g.err, err);
        return;
    }

    // this lane's dims: two words of a head
    const int32_t pairs = a.rot_dim / 2, twos = a.interleaved ? 0 : pairs / 8;
    const int32_t unit = lane % LANES;
    const bool active = unit * 16 < dim, two = unit < twos;
    const int32_t d0 = active ? (two ? unit * 8 : unit * 16) : 0;
    const int32_t d1 = two ? d0 + pairs : d0 + 8;
    const int32_t q_heads = a.q ? g.q_heads : 0, heads = q_heads + g.kv_heads;
    const int64_t r = (int64_t)b * g.rows + t;
    struct Words {
        Eight<T> u, v;
    };
    const auto fetch = [&](int32_t h) {
        const T *from = h < q_heads ? (const T *)a.q + r * a.q_stride + (int64_t)h * dim
                                    : (const T *)a.k + r * a.kv_stride +
                                          (int64_t)(h - q_heads) * dim;
        return Words{load8(from + d0), load8(from + d1)};
    };
    // the first heads are on their way before the depth and the angles
    int32_t h = lane / LANES;
    Words next{};
    if (active && h < heads)
        next = fetch(h);

    int32_t depth = t;
    if (ta.parent) {
        if (tree.load(ta.parent, g, b, lane)) {
            if (t == 0 && lane == 0)
                atomicOr(g.err, (uint32_t)kErrBlock);
            return;
        }
        depth = tree.depth(t);
    }
    const int32_t cell = length - 1 + t, page = page_of(g, b, cell);
    if (page < 0 && lane == 0)
        atomicOr(g.err, (uint32_t)kErrPage);
    float2 *cs = (float2 *)lds + wave * kMaxPairs;
    for (int32_t i = lane; i < pairs; i += kWave) {
        float c, s;
        turn(a.turns[i], length - 1 + depth, a.magnitude, c, s);
        cs[i] = float2{c, s};
    }
    // (the wavefront's own words, read by other lanes after they are written)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const bool turn0 = two || (a.interleaved && d0 < a.rot_dim);
    const bool turn1 = two || (a.interleaved && d1 < a.rot_dim);
    // The eight pairs: of d0 + k and d1 + k, or of the words one after the other.
    float2 m[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const bool turns = k < 4 ? turn0 : turn1;
        m[k] = turns ? cs[two ? d0 + k : d0 / 2 + k] : float2{1.0f, 0.0f};
    }

    for (int32_t base = 0; base < heads; base += kWave / LANES, h += kWave / LANES) {
        const Words x = next;
        if (active && h + kWave / LANES < heads)
            next = fetch(h + kWave / LANES);
        const bool is_q = h < q_heads;
        const float *weight = is_q ? ta.q_norm : ta.k_norm;
        float y[8], z[8], sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            y[k] = to_f32(x.u.x[k]);
            z[k] = to_f32(x.v.x[k]);
            sum = fmaf(y[k], y[k], fmaf(z[k], z[k], sum));
        }
        sum = lanes_sum<LANES>(active ? sum : 0.0f);
        if (!active || h >= heads)
            continue;
        if (weight) {
            // (read again for each head: held, they would cost a quarter of the
            // wavefronts, 22.6 us against 19.8 for 64 trees of up to 64 rows)
            const Weights w0 = *(const Weights *)(weight + d0);
            const Weights w1 = *(const Weights *)(weight + d1);
            const float f = norm_of(sum, dim, ta.eps);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                y[k] *= f * w0.x[k];
                z[k] *= f * w1.x[k];
            }
        }
        if (two) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float e = y[k], f = z[k];
                y[k] = e * m[k].x - f * m[k].y;
                z[k] = e * m[k].y + f * m[k].x;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float e = y[2 * k], f = y[2 * k + 1], i = z[2 * k], j = z[2 * k + 1];
                if (turn0) {
                    y[2 * k] = e * m[k].x - f * m[k].y;
                    y[2 * k + 1] = e * m[k].y + f * m[k].x;
                }
                if (turn1) {
                    z[2 * k] = i * m[4 + k].x - j * m[4 + k].y;
                    z[2 * k + 1] = i * m[4 + k].y + j * m[4 + k].x;
                }
            }
        }
        if (is_q) {
            T *out = (T *)a.out_q + (r * g.q_heads + h) * dim;
            store8<T>(out + d0, y);
            store8<T>(out + d1, z);
        } else if (page >= 0) {
            const int32_t kh = h - q_heads;
            if (g.k_scale) {
                const float scale = g.k_scale[kh];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    y[k] /= scale;
                    z[k] /= scale;
                }
            }
            C *out = (C *)a.k_cache +
                     (((int64_t)page * g.kv_heads + kh) * tokens + (cell & (tokens - 1))) * dim;
            store8<C>(out + d0, y);
            store8<C>(out + d1, z);
        }
    }
}

// Any alignment and any part of a head: one workgroup per row, a wavefront a
// head, an element or a pair a lane.
template <typename T, typename C>
__global__ __launch_bounds__(kThreads) void tree_elements(TreeAppendArgs ta)
{
    const KvAppendArgs &a = ta.kv;
    const BlockArgs &g = a.blk;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
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
    int32_t depth = t;
    if (ta.parent) {
        WaveTree tree;
        if (tree.load(ta.parent, g, b, lane)) {
            if (t == 0 && threadIdx.x == 0)
                atomicOr(g.err, (uint32_t)kErrBlock);
            return;
        }
        depth = tree.depth(t);
    }
    const int32_t cell = length - 1 + t, page = page_of(g, b, cell);
    if (page < 0 && threadIdx.x == 0)
        atomicOr(g.err, (uint32_t)kErrPage);
    const int32_t dim = g.head_dim, half = a.rot_dim / 2, tokens = 1 << g.page_shift;
    const int32_t slot = cell & (tokens - 1), q_heads = a.q ? g.q_heads : 0;
    const int64_t r = (int64_t)b * g.rows + t;
    for (int32_t h = wave; h < q_heads + g.kv_heads; h += kWaves) {
        const bool is_q = h < q_heads;
        const int32_t kh = h - q_heads;
        const T *x = is_q ? (const T *)a.q + r * a.q_stride + (int64_t)h * dim
                          : (const T *)a.k + r * a.kv_stride + (int64_t)kh * dim;
        const float *weight = is_q ? ta.q_norm : ta.k_norm;
        float sum = 0.0f;
        for (int32_t d = lane; d < dim; d += kWave) {
            const float y = to_f32(x[d]);
            sum = fmaf(y, y, sum);
        }
        // (also: every lane has read its part before q is rotated in place)
        const float f = norm_of(lanes_sum<kWave>(sum), dim, ta.eps);
        for (int32_t e = lane; e < dim - half; e += kWave) {
            const bool two = e < half;
            const int32_t d = two ? (a.interleaved ? 2 * e : e) : e + half;
            const int32_t d2 = two ? (a.interleaved ? d + 1 : d + half) : d;
            float y = to_f32(x[d]), z = to_f32(x[d2]);
            if (weight) {
                y *= f * weight[d];
                z *= f * weight[d2];
            }
            if (two) {
                float c, s;
                turn(a.turns[e], length - 1 + depth, a.magnitude, c, s);
                const float y0 = y;
                y = y0 * c - z * s;
                z = y0 * s + z * c;
            }
            if (is_q) {
                T *out = (T *)a.out_q + (r * g.q_heads + h) * dim;
                out[d] = from_f32<T>(y);
                if (two)
                    out[d2] = from_f32<T>(z);
            } else if (page >= 0) {
                const float scale = g.k_scale ? g.k_scale[kh] : 1.0f;
                C *out =
                    (C *)a.k_cache + (((int64_t)page * g.kv_heads + kh) * tokens + slot) * dim;
                out[d] = from_f32<C>(y / scale);
                if (two)
                    out[d2] = from_f32<C>(z / scale);
            }
        }
    }
    if (page < 0)
        return;
    for (int32_t i = threadIdx.x; i < g.kv_heads * dim; i += kThreads) {
        const float scale = g.v_scale ? g.v_scale[i / dim] : 1.0f;
        ((C *)a.v_cache)[((int64_t)page * g.kv_heads * dim + i) * tokens + slot] =
            from_f32<C>(to_f32(((const T *)a.v)[r * a.kv_stride + i]) / scale);
    }
}

template <typename T, typename C>
hipError_t launch_cells(const TreeAppendArgs &ta, hipStream_t s)
{
    const KvAppendArgs &a = ta.kv;
    const BlockArgs &g = a.blk;
    const bool words = !(((uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.out_q) &
                         15u) &&
                       !((a.q ? a.q_stride : 0) & 7) && !(a.kv_stride & 7) &&
                       a.rot_dim % (a.interleaved ? 8 : 16) == 0;
    if (!words) {
        const int64_t rows = (int64_t)g.batch * g.rows;
        if (!fits_grid(rows, kThreads))
            return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((tree_elements<T, C>), dim3((uint32_t)rows), dim3(kThreads), 0, s, ta);
        return hipGetLastError();
    }
    const int64_t turning = (int64_t)g.batch * ((g.rows + kWaves - 1) / kWaves);
    const int64_t tiles = (g.rows + kSpan - 2) / kSpan + 1;
    const int64_t storing = (int64_t)g.batch * g.kv_heads * tiles;
    if (!fits_grid(turning + storing, kThreads))
        return hipErrorInvalidConfiguration;
    const size_t turn_lds = (size_t)kWaves * kMaxPairs * sizeof(float2);
    const size_t tile_lds = (size_t)kSpan * (g.head_dim + kPad) * sizeof(T);
    const size_t lds = turn_lds > tile_lds ? turn_lds : tile_lds;
    const dim3 grid((uint32_t)(turning + storing));
    const auto start = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), lds, s, ta, (uint32_t)turning,
                           (uint32_t)tiles);
    };
    if (g.head_dim <= 64)
        start(tree_words<T, C, 4>);
    else if (g.head_dim <= 128)
        start(tree_words<T, C, 8>);
    else
        start(tree_words<T, C, 16>);
    return hipGetLastError();
}

// One wavefront per request, layer and kv head. Path nodes rise, so a move's
// target is never the source of a later move: the moves of a batch are loaded
// before any of them is stored, batch after batch. Of V, whose positions lie
// side by side, kBatch moves of a dim are neighbouring lanes: they touch the
// same line.
// Bound by V's lines: a moved cell is 2 bytes of a 128-byte line in every dim. 64
// requests, 32 layers, 8 kv heads of 128, paths of up to 8 nodes: 118 us, 142 to 154
// when the cache was not just used, for 334 MB read and 78 MB written where the moved
// cells are 67 MB. K alone 14 us, with V's stores 33, with V's loads 73. Non-temporal
// loads: 128; stores too: 153.
template <typename C, int D>
__global__ __launch_bounds__(kThreads) void keep_cells(KeepArgs a, int64_t units)
{
    constexpr int kBatch = 8, kSide = kWave / kBatch;
    constexpr int kWord = 16 / sizeof(C);  // cells of a word
    const BlockArgs &g = a.blk;
    const int lane = threadIdx.x % kWave;
    const int64_t id = (int64_t)blockIdx.x * kWaves +
                       __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (id >= units)
        return;
    const int32_t h = (int32_t)(id % g.kv_heads);
    const int64_t rest = id / g.kv_heads;
    const int32_t layer = (int32_t)(rest % a.layers), b = (int32_t)(rest / a.layers);
    const bool tells = h == 0 && layer == 0 && lane == 0;
    int32_t length;
    uint32_t err;
    const int32_t n = block_rows(g, b, length, err);
    if (n <= 0) {
        if (err && tells)
            atomicOr(g.err, err);
        return;
    }
    // the whole path is checked first: a bad one moves nothing
    const int32_t moves = a.accepted[b];
    if (moves == 0)
        return;
    const int32_t *path = a.path + (int64_t)b * g.rows;
    bool bad = moves < 0 || moves >= n, page = false;
    int32_t first = moves + 1;  // the first move that has to be made
    if (!bad)
        for (int32_t i = lane; i <= moves; i += kWave) {
            const int32_t node = path[i], before = i ? path[i - 1] : -1;
            const bool fine = (i ? node > before : node == 0) && node < n && before < n;
            bad |= !fine;
            if (fine && node != i) {
                first = i < first ? i : first;
                page |= page_of(g, b, length - 1 + node) < 0 ||
                        page_of(g, b, length - 1 + i) < 0;
            }
        }
    bad = __any(bad);
    page = __any(page);
    if (bad || page) {
        if (tells)
            atomicOr(g.err, (bad ? (uint32_t)kErrBlock : 0u) | (page ? (uint32_t)kErrPage : 0u));
        return;
    }
    for (int i = kWave / 2; i; i >>= 1) {
        const int32_t y = __shfl_xor(first, i);
        first = y < first ? y : first;
    }

    constexpr int kKeys = (D / kWord + kSide - 1) / kSide, kValues = D / kSide;
    const int32_t tokens = 1 << g.page_shift;
    C *const kc = (C *)a.k_cache + layer * a.k_layer;
    C *const vc = (C *)a.v_cache + layer * a.v_layer;
    const int32_t side = lane / kBatch;
    for (int32_t at = first; at <= moves; at += kBatch) {
        // this lane's move
        const int32_t i = at + lane % kBatch;
        const bool live = i <= moves;
        const int32_t from = length - 1 + path[live ? i : moves], to = length - 1 + (live ? i : moves);
        const int64_t from_page = page_of(g, b, from), to_page = page_of(g, b, to);
        const int64_t src = (from_page * g.kv_heads + h) * tokens * D;
        const int64_t dst = (to_page * g.kv_heads + h) * tokens * D;
        const int32_t src_at = from & (tokens - 1), dst_at = to & (tokens - 1);
        U4 k[kKeys];
        C v[kValues];
#pragma unroll
        for (int w = 0; w < kKeys; ++w) {
            const int32_t d = (w * kSide + side) * kWord;
            if (live && d < D)
                k[w] = *(const U4 *)(kc + src + (int64_t)src_at * D + d);
        }
#pragma unroll
        for (int w = 0; w < kValues; ++w) {
            const int32_t d = w * kSide + side;
            if (live)
                v[w] = vc[src + (int64_t)d * tokens + src_at];
        }
        // (every lane's loads have come before a store leaves)
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int w = 0; w < kKeys; ++w) {
            const int32_t d = (w * kSide + side) * kWord;
            if (live && d < D)
                *(U4 *)(kc + dst + (int64_t)dst_at * D + d) = k[w];
        }
#pragma unroll
        for (int w = 0; w < kValues; ++w) {
            const int32_t d = w * kSide + side;
            if (live)
                vc[dst + (int64_t)d * tokens + dst_at] = v[w];
        }
    }
}

template <typename C>
hipError_t launch_keep(const KeepArgs &a, hipStream_t s)
{
    const int64_t units = (int64_t)a.blk.batch * a.layers * a.blk.kv_heads;
    const int64_t groups = (units + kWaves - 1) / kWaves;
    if (!fits_grid(groups, kThreads))
        return hipErrorInvalidConfiguration;
    const auto start = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((uint32_t)groups), dim3(kThreads), 0, s, a, units);
    };
    switch (a.blk.head_dim) {
    case 64: start(keep_cells<C, 64>); break;
    case 96: start(keep_cells<C, 96>); break;
    case 128: start(keep_cells<C, 128>); break;
    case 192: start(keep_cells<C, 192>); break;
    default: start(keep_cells<C, 256>); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append_tree(const TreeAppendArgs &a, hipStream_t s)
{
    const BlockArgs &g = a.kv.blk;
    const bool wide = g.cache_dtype != PLD_E4M3;
    if (g.dtype == PLD_BF16)
        return wide ? launch_cells<__bf16, __bf16>(a, s) : launch_cells<__bf16, E4m3>(a, s);
    return wide ? launch_cells<_Float16, _Float16>(a, s) : launch_cells<_Float16, E4m3>(a, s);
}

// (cells are moved as they are: two kinds by their size)
hipError_t launch_kv_keep(const KeepArgs &a, hipStream_t s)
{
    return a.blk.cache_dtype == PLD_E4M3 ? launch_keep<uint8_t>(a, s) : launch_keep<uint16_t>(a, s);
}

}  // namespace pld
