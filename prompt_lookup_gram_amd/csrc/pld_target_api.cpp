// C-ABI entry points of the verify step (include/pld.h): the target context,
// argument checks and the launches of pld_kv.hip, pld_attend.hip,
// pld_verify.hip and their counterparts for trees. No compute happens here but
// the rotary frequencies, once per context.

#include <math.h>
#include <stdint.h>
#include <string.h>

#include <new>

#include <hip/hip_runtime_api.h>

#include "pld.h"
#include "pld_ctx.h"
#include "pld_target.h"

using pld::fail;
using pld::hip_fail;

namespace pld {

void target_release(Target *t)
{
    if (t->turns) (void)hipFree(t->turns);
    if (t->verify_ws) (void)hipFree(t->verify_ws);
    if (t->attend_ws) (void)hipFree(t->attend_ws);
    delete t;
}

}  // namespace pld

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr int kMaxPairs = 128;  // head_dim 256
constexpr int64_t kMost = 1 << 30;
constexpr int32_t kMaxVocab = 1 << 24;

// Turns (angle / 2 pi) per position of each rotated pair, in 64 bits.
void rope_turns(const pld_rope_params &r, double *turns)
{
    const int32_t n = r.rot_dim;
    double lo = 0.0, hi = 0.0;
    if (r.scaling == PLD_ROPE_BANDED && n > 0) {
        // the pair whose wavelength fits beta times into original_len
        const double lb = log(r.base);
        lo = floor(n * 0.5 * log(r.original_len / (r.beta_fast * kTwoPi)) / lb);
        hi = ceil(n * 0.5 * log(r.original_len / (r.beta_slow * kTwoPi)) / lb);
        lo = lo < 0.0 ? 0.0 : lo;
        hi = hi > n - 1.0 ? n - 1.0 : hi;
    }
    for (int32_t i = 0; i < n / 2; ++i) {
        double f = pow(r.base, -2.0 * i / n);
        if (r.scaling == PLD_ROPE_LINEAR) {
            f /= r.factor;
        } else if (r.scaling == PLD_ROPE_BANDED) {
            const double span = hi - lo > 0.001 ? hi - lo : 0.001;
            double ramp = (i - lo) / span;
            ramp = ramp < 0.0 ? 0.0 : (ramp > 1.0 ? 1.0 : ramp);
            f = f / r.factor * ramp + f * (1.0 - ramp);
        }
        turns[i] = f / kTwoPi;
    }
}

bool positive(double x) { return x > 0.0 && isfinite(x); }

pld_status check_params(const pld_target_params &p)
{
    if (p.max_batch < 1)
        return fail(PLD_EINVAL, "max_batch must be >= 1 (got %d)", p.max_batch);
    if (p.max_rows < 1)
        return fail(PLD_EINVAL, "max_rows must be >= 1 (got %d)", p.max_rows);
    // (the kernels step past the last position, row and logit in 32 bits)
    if (p.max_len < 1 || p.max_len > kMost)
        return fail(PLD_EINVAL, "max_len must be in [1, 2^30] (got %lld)", (long long)p.max_len);
    if ((int64_t)p.max_batch * p.max_rows > kMost)
        return fail(PLD_EINVAL, "max_batch * max_rows must be at most 2^30");
    if (p.vocab < 0 || p.vocab > kMaxVocab)
        return fail(PLD_EINVAL, "vocab must be in [0, 2^24] (got %d)", p.vocab);
    if (p.q_heads < 0 || p.kv_heads < 0 || (p.q_heads == 0) != (p.kv_heads == 0) ||
        (p.kv_heads > 0 && p.q_heads % p.kv_heads != 0) || p.q_heads > 65536)
        return fail(PLD_EINVAL, "q_heads must be a multiple of kv_heads, at most 65536 "
                    "(got %d, %d)", p.q_heads, p.kv_heads);
    if (p.q_heads == 0 && p.vocab == 0)
        return fail(PLD_EINVAL, "a target context needs heads or a vocab");
    if (p.q_heads == 0)
        return PLD_OK;
    if ((int64_t)p.max_rows * (p.q_heads / p.kv_heads) > kMost)
        return fail(PLD_EINVAL, "max_rows * q_heads / kv_heads must be at most 2^30");
    if (p.head_dim != 64 && p.head_dim != 96 && p.head_dim != 128 && p.head_dim != 192 &&
        p.head_dim != 256)
        return fail(PLD_EINVAL, "head_dim %d not one of 64, 96, 128, 192, 256", p.head_dim);
    if (p.dtype != PLD_F16 && p.dtype != PLD_BF16)
        return fail(PLD_EINVAL, "dtype must be PLD_F16 or PLD_BF16 (got %d)", p.dtype);
    if (p.cache_dtype != p.dtype && p.cache_dtype != PLD_E4M3)
        return fail(PLD_EINVAL, "cache_dtype must be dtype or PLD_E4M3 (got %d)", p.cache_dtype);
    if (p.page_tokens != 16 && p.page_tokens != 32 && p.page_tokens != 64 &&
        p.page_tokens != 128 && p.page_tokens != 256)
        return fail(PLD_EINVAL, "page_tokens %d not one of 16, 32, 64, 128, 256", p.page_tokens);
    const pld_rope_params &r = p.rope;
    if (r.rot_dim < 0 || r.rot_dim > p.head_dim || (r.rot_dim & 1))
        return fail(PLD_EINVAL, "rope.rot_dim must be even, in [0, head_dim] (got %d)", r.rot_dim);
    if (r.rot_dim == 0)
        return PLD_OK;
    if (r.interleaved != 0 && r.interleaved != 1)
        return fail(PLD_EINVAL, "rope.interleaved must be 0 or 1 (got %d)", r.interleaved);
    if (r.scaling < PLD_ROPE_PLAIN || r.scaling > PLD_ROPE_BANDED)
        return fail(PLD_EINVAL, "rope.scaling must be PLD_ROPE_* (got %d)", r.scaling);
    if (!(r.base > 1.0) || !isfinite(r.base) || !positive(r.magnitude))
        return fail(PLD_EINVAL, "need rope.base > 1 and rope.magnitude > 0, finite");
    if (r.scaling != PLD_ROPE_PLAIN && !positive(r.factor))
        return fail(PLD_EINVAL, "need rope.factor > 0, finite");
    if (r.scaling == PLD_ROPE_BANDED &&
        (r.original_len < 1 || !positive(r.beta_fast) || !positive(r.beta_slow) ||
         r.beta_fast < r.beta_slow))
        return fail(PLD_EINVAL, "need rope.original_len >= 1 and beta_fast >= beta_slow > 0");
    return PLD_OK;
}

// The common checks of a call on a target context.
pld_status check_call(pld_ctx *ctx, int32_t rows, int32_t batch)
{
    if (!ctx)
        return fail(PLD_EINVAL, "ctx is null");
    if (!ctx->target)
        return fail(PLD_EINVAL, "not a target context (see pld_create_target)");
    const pld_target_params &p = ctx->target->p;
    if (rows < 1 || rows > p.max_rows)
        return fail(PLD_EINVAL, "rows %d outside [1, max_rows=%d]", rows, p.max_rows);
    if (batch < 0 || batch > p.max_batch)
        return fail(PLD_EINVAL, "batch %d outside [0, max_batch=%d]", batch, p.max_batch);
    int device = -1;
    const hipError_t e = batch > 0 ? hipGetDevice(&device) : hipSuccess;
    if (e != hipSuccess)
        return hip_fail(e, "hipGetDevice");
    if (batch > 0 && device != ctx->device)
        return fail(PLD_EINVAL, "the context belongs to device %d, the current device is %d",
                    ctx->device, device);
    return PLD_OK;
}

// The checks on a batch's blocks and the cache they stand in; fills `blk`.
pld_status block_args(pld_ctx *ctx, int32_t rows, const int32_t *lengths,
                      const int32_t *draft_len, int64_t max_len, int32_t batch,
                      const int32_t *page_table, int64_t table_stride, const void *k_cache,
                      const void *v_cache, int64_t n_pages, const float *k_scale,
                      const float *v_scale, pld::BlockArgs &blk)
{
    pld_status st = check_call(ctx, rows, batch);
    if (st != PLD_OK)
        return st;
    const pld_target_params &p = ctx->target->p;
    if (p.q_heads == 0)
        return fail(PLD_EINVAL, "the context has no heads (see pld_target_params)");
    if (max_len < 0 || max_len > p.max_len)
        return fail(PLD_EINVAL, "max_len %lld outside [0, the context's %lld]",
                    (long long)max_len, (long long)p.max_len);
    if (n_pages < 1 || n_pages > 0x7fffffffLL)
        return fail(PLD_EINVAL, "n_pages must be in [1, 2^31-1] (got %lld)", (long long)n_pages);
    if (table_stride < 1)
        return fail(PLD_EINVAL, "table_stride must be >= 1 (got %lld)", (long long)table_stride);
    if (batch > 0 && (!lengths || !draft_len || !page_table || !k_cache || !v_cache))
        return fail(PLD_EINVAL, "null buffer pointer");
    if (((uintptr_t)lengths | (uintptr_t)draft_len | (uintptr_t)page_table | (uintptr_t)k_scale |
         (uintptr_t)v_scale) & 3u)
        return fail(PLD_EINVAL, "int32 and float buffers must be 4-byte aligned");
    if (((uintptr_t)k_cache | (uintptr_t)v_cache) & 15u)
        return fail(PLD_EINVAL, "k_cache and v_cache must be 16-byte aligned");
    memset(&blk, 0, sizeof(blk));
    blk.lengths = lengths;
    blk.draft_len = draft_len;
    blk.rows = rows;
    blk.batch = batch;
    blk.max_len = (int32_t)(max_len ? max_len : p.max_len);
    blk.table = page_table;
    blk.table_stride = table_stride;
    blk.n_pages = n_pages;
    blk.page_shift = ctx->target->page_shift;
    blk.q_heads = p.q_heads;
    blk.kv_heads = p.kv_heads;
    blk.head_dim = p.head_dim;
    blk.dtype = p.dtype;
    blk.cache_dtype = p.cache_dtype;
    blk.k_scale = p.cache_dtype == PLD_E4M3 ? k_scale : nullptr;
    blk.v_scale = p.cache_dtype == PLD_E4M3 ? v_scale : nullptr;
    blk.err = ctx->err;
    return PLD_OK;
}

// The checks of a cache append; fills `a`.
pld_status append_args(pld_ctx *ctx, const void *q, int64_t q_stride, const void *k,
                       const void *v, int64_t kv_stride, int32_t rows, const int32_t *lengths,
                       const int32_t *draft_len, int32_t batch, const int32_t *page_table,
                       int64_t table_stride, void *k_cache, void *v_cache, int64_t n_pages,
                       const float *k_scale, const float *v_scale, void *out_q,
                       pld::KvAppendArgs &a)
{
    pld_status st = block_args(ctx, rows, lengths, draft_len, 0, batch, page_table, table_stride,
                               k_cache, v_cache, n_pages, k_scale, v_scale, a.blk);
    if (st != PLD_OK)
        return st;
    const pld_target_params &p = ctx->target->p;
    const int64_t q_width = (int64_t)p.q_heads * p.head_dim;
    const int64_t kv_width = (int64_t)p.kv_heads * p.head_dim;
    if (batch > 0 && (!k || !v || (q != nullptr) != (out_q != nullptr)))
        return fail(PLD_EINVAL, "k or v is null, or only one of q and out_q is");
    if ((q && q_stride < q_width) || kv_stride < kv_width)
        return fail(PLD_EINVAL, "q_stride and kv_stride must hold a row (%lld and %lld elements)",
                    (long long)q_width, (long long)kv_width);
    if (q && q == out_q && q_stride != q_width)
        return fail(PLD_EINVAL, "q rotated in place needs q_stride %lld", (long long)q_width);
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out_q) & 1u)
        return fail(PLD_EINVAL, "q, k, v and out_q must be 2-byte aligned");
    a.q = q;
    a.q_stride = q_stride;
    a.k = k;
    a.v = v;
    a.kv_stride = kv_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.out_q = out_q;
    a.turns = ctx->target->turns;
    a.rot_dim = p.rope.rot_dim;
    a.interleaved = p.rope.interleaved;
    a.magnitude = (float)p.rope.magnitude;
    return PLD_OK;
}

// The checks of an attention; fills `a`.
pld_status attend_args(pld_ctx *ctx, const void *q, int64_t q_stride, int32_t rows,
                       const int32_t *lengths, const int32_t *draft_len, int64_t max_len,
                       int32_t batch, const int32_t *page_table, int64_t table_stride,
                       const void *k_cache, const void *v_cache, int64_t n_pages,
                       const float *k_scale, const float *v_scale, float scale, int32_t window,
                       void *out, float *out_lse, pld::AttendArgs &a)
{
    pld_status st = block_args(ctx, rows, lengths, draft_len, max_len, batch, page_table,
                               table_stride, k_cache, v_cache, n_pages, k_scale, v_scale, a.blk);
    if (st != PLD_OK)
        return st;
    const pld_target_params &p = ctx->target->p;
    if (batch > 0 && (!q || !out))
        return fail(PLD_EINVAL, "null buffer pointer");
    if (q_stride < (int64_t)p.q_heads * p.head_dim || (q_stride & 7))
        return fail(PLD_EINVAL, "q_stride must be a multiple of 8 elements and hold a row "
                    "(got %lld)", (long long)q_stride);
    if (((uintptr_t)q | (uintptr_t)out) & 15u)
        return fail(PLD_EINVAL, "q and out must be 16-byte aligned");
    if (q && q == out && q_stride != (int64_t)p.q_heads * p.head_dim)
        return fail(PLD_EINVAL, "out in q's place needs q_stride %lld",
                    (long long)p.q_heads * p.head_dim);
    if ((uintptr_t)out_lse & 3u)
        return fail(PLD_EINVAL, "out_lse must be 4-byte aligned");
    if (!isfinite(scale))
        return fail(PLD_EINVAL, "scale must be finite");
    if (window < 0)
        return fail(PLD_EINVAL, "window must be >= 0 (got %d)", window);
    a.q = q;
    a.q_stride = q_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.scale = scale != 0.0f ? scale : (float)(1.0 / sqrt((double)p.head_dim));
    a.window = window;
    a.out = out;
    a.out_lse = out_lse;
    a.ws = ctx->target->attend_ws;
    a.ws_rows = ctx->target->attend_rows;
    a.parent = nullptr;
    return PLD_OK;
}

// The checks of a verification; fills `a`.
pld_status verify_args(pld_ctx *ctx, const void *logits, int32_t logits_dtype,
                       int64_t logits_stride, int32_t rows, const int32_t *draft,
                       const int32_t *draft_len, const uint64_t *src, const float *draft_probs,
                       int32_t head, const float *temperature, const float *uniform,
                       int32_t batch, int32_t *out_tokens, int32_t *out_accepted,
                       int32_t *out_counts, float *out_logprobs, pld::VerifyArgs &a)
{
    pld_status st = check_call(ctx, rows, batch);
    if (st != PLD_OK)
        return st;
    const pld_target_params &p = ctx->target->p;
    if (p.vocab == 0)
        return fail(PLD_EINVAL, "the context has no vocab (see pld_target_params)");
    if (logits_dtype != PLD_F32 && logits_dtype != PLD_F16 && logits_dtype != PLD_BF16)
        return fail(PLD_EINVAL, "logits_dtype must be PLD_F32, PLD_F16 or PLD_BF16 (got %d)",
                    logits_dtype);
    if (logits_stride < p.vocab)
        return fail(PLD_EINVAL, "logits_stride %lld below the vocab %d", (long long)logits_stride,
                    p.vocab);
    if (head < 0 || head > rows - 1 || (head > 0) != (draft_probs != nullptr))
        return fail(PLD_EINVAL, "head must be in [0, rows - 1], and > 0 exactly with draft_probs "
                    "(got %d)", head);
    if (batch > 0 && (!logits || !draft_len || !uniform || !out_tokens || !out_accepted ||
                      !out_counts || (rows > 1 && !draft)))
        return fail(PLD_EINVAL, "null buffer pointer");
    if (((uintptr_t)draft | (uintptr_t)draft_len | (uintptr_t)draft_probs |
         (uintptr_t)temperature | (uintptr_t)uniform | (uintptr_t)out_tokens |
         (uintptr_t)out_accepted | (uintptr_t)out_counts | (uintptr_t)out_logprobs) & 3u)
        return fail(PLD_EINVAL, "int32 and float buffers must be 4-byte aligned");
    if ((uintptr_t)src & 7u)
        return fail(PLD_EINVAL, "src must be 8-byte aligned");
    if ((uintptr_t)logits & (logits_dtype == PLD_F32 ? 3u : 1u))
        return fail(PLD_EINVAL, "logits must be aligned to their elements");
    a.logits = logits;
    a.dtype = logits_dtype;
    a.stride = logits_stride;
    a.rows = rows;
    a.batch = batch;
    a.vocab = p.vocab;
    a.draft = draft;
    a.draft_len = draft_len;
    a.src = src;
    a.probs = draft_probs;
    a.head = head;
    a.temperature = temperature;
    a.uniform = uniform;
    a.out_tokens = out_tokens;
    a.out_accepted = out_accepted;
    a.out_counts = out_counts;
    a.out_logprobs = out_logprobs;
    a.err = ctx->err;
    a.stats = ctx->target->verify_ws;
    a.max_batch = p.max_batch;
    a.max_rows = p.max_rows;
    return PLD_OK;
}

// The checks that a tree's calls add.
pld_status tree_rows(int32_t rows, const int32_t *parent)
{
    if (rows > PLD_TREE_ROWS)
        return fail(PLD_EINVAL, "rows %d: a tree has at most %d", rows, PLD_TREE_ROWS);
    if ((uintptr_t)parent & 3u)
        return fail(PLD_EINVAL, "parent must be 4-byte aligned");
    return PLD_OK;
}

}  // namespace

extern "C" {

pld_status pld_target_params_default(pld_target_params *params)
{
    if (!params)
        return fail(PLD_EINVAL, "params is null");
    memset(params, 0, sizeof(*params));
    params->max_batch = 1;
    params->max_rows = 16;
    params->max_len = 32768;
    params->head_dim = 128;
    params->dtype = PLD_BF16;
    params->cache_dtype = PLD_BF16;
    params->page_tokens = 64;
    params->rope.original_len = 32768;
    params->rope.base = 10000.0;
    params->rope.factor = 1.0;
    params->rope.beta_fast = 32.0;
    params->rope.beta_slow = 1.0;
    params->rope.magnitude = 1.0;
    return PLD_OK;
}

pld_status pld_create_target(pld_ctx **out, const pld_target_params *params, hipStream_t stream)
{
    if (!out || !params)
        return fail(PLD_EINVAL, "out or params is null");
    pld_status st = check_params(*params);
    if (st != PLD_OK)
        return st;
    const pld_target_params &p = *params;
    pld_ctx *c = nullptr;
    st = pld_create(&c, p.max_batch, p.max_len, 0, stream);
    if (st != PLD_OK)
        return st;
    pld::Target *t = new (std::nothrow) pld::Target();
    if (!t) {
        (void)pld_destroy(c);
        return fail(PLD_ENOMEM, "host allocation failed");
    }
    memset(t, 0, sizeof(*t));
    c->target = t;
    t->p = p;
    for (int32_t n = p.page_tokens; n > 1; n >>= 1)
        ++t->page_shift;
    double turns[kMaxPairs];
    const int32_t pairs = p.q_heads > 0 ? p.rope.rot_dim / 2 : 0;
    hipError_t e = hipSuccess;
    bool memory = true;
    if (pairs > 0) {
        rope_turns(p.rope, turns);
        memory = hipMalloc((void **)&t->turns, pairs * sizeof(double)) == hipSuccess;
        if (memory)
            e = hipMemcpyAsync(t->turns, turns, pairs * sizeof(double), hipMemcpyHostToDevice,
                               stream);
        // the copy's source is this frame's: wait before leaving it
        const hipError_t w = hipStreamSynchronize(stream);
        if (e == hipSuccess)
            e = w;
    }
    if (memory && e == hipSuccess && p.vocab > 0)
        memory = hipMalloc(&t->verify_ws, pld::verify_workspace(p.max_batch, p.max_rows,
                                                                p.vocab)) == hipSuccess;
    if (memory && e == hipSuccess && p.vocab > 0) {
        e = pld::verify_clear(t->verify_ws, p.max_batch, p.max_rows, p.vocab, stream);
        const hipError_t w = hipStreamSynchronize(stream);
        if (e == hipSuccess)
            e = w;
    }
    if (memory && e == hipSuccess && p.q_heads > 0) {
        t->attend_rows = pld::attend_rows(p);
        memory = hipMalloc((void **)&t->attend_ws,
                           (size_t)t->attend_rows * (p.head_dim + 2) * sizeof(float)) == hipSuccess;
    }
    if (!memory || e != hipSuccess) {
        (void)hipGetLastError();
        (void)pld_destroy(c);
        return memory ? hip_fail(e, "target context initialisation")
                      : fail(PLD_ENOMEM, "device allocation of the verify workspaces failed");
    }
    *out = c;
    return PLD_OK;
}

pld_status pld_kv_append(pld_ctx *ctx, const void *q, int64_t q_stride, const void *k,
                         const void *v, int64_t kv_stride, int32_t rows,
                         const int32_t *lengths, const int32_t *draft_len, int32_t batch,
                         const int32_t *page_table, int64_t table_stride, void *k_cache,
                         void *v_cache, int64_t n_pages, const float *k_scale,
                         const float *v_scale, void *out_q, hipStream_t stream)
{
    pld::KvAppendArgs a;
    const pld_status st =
        append_args(ctx, q, q_stride, k, v, kv_stride, rows, lengths, draft_len, batch, page_table,
                    table_stride, k_cache, v_cache, n_pages, k_scale, v_scale, out_q, a);
    if (st != PLD_OK || batch == 0)
        return st;
    const hipError_t e = pld::launch_kv_append(a, stream);
    if (e != hipSuccess)
        return hip_fail(e, "cache append launch");
    return PLD_OK;
}

pld_status pld_attend(pld_ctx *ctx, const void *q, int64_t q_stride, int32_t rows,
                      const int32_t *lengths, const int32_t *draft_len, int64_t max_len,
                      int32_t batch, const int32_t *page_table, int64_t table_stride,
                      const void *k_cache, const void *v_cache, int64_t n_pages,
                      const float *k_scale, const float *v_scale, float scale, int32_t window,
                      void *out, float *out_lse, hipStream_t stream)
{
    pld::AttendArgs a;
    const pld_status st =
        attend_args(ctx, q, q_stride, rows, lengths, draft_len, max_len, batch, page_table,
                    table_stride, k_cache, v_cache, n_pages, k_scale, v_scale, scale, window, out,
                    out_lse, a);
    if (st != PLD_OK || batch == 0)
        return st;
    const hipError_t e = pld::launch_attend(a, stream);
    if (e != hipSuccess)
        return hip_fail(e, "attention launch");
    return PLD_OK;
}

pld_status pld_verify(pld_ctx *ctx, const void *logits, int32_t logits_dtype,
                      int64_t logits_stride, int32_t rows, const int32_t *draft,
                      const int32_t *draft_len, const uint64_t *src, const float *draft_probs,
                      int32_t head, const float *temperature, const float *uniform,
                      int32_t batch, int32_t *out_tokens, int32_t *out_accepted,
                      int32_t *out_counts, float *out_logprobs, hipStream_t stream)
{
    pld::VerifyArgs a;
    const pld_status st =
        verify_args(ctx, logits, logits_dtype, logits_stride, rows, draft, draft_len, src,
                    draft_probs, head, temperature, uniform, batch, out_tokens, out_accepted,
                    out_counts, out_logprobs, a);
    if (st != PLD_OK || batch == 0)
        return st;
    const hipError_t e = pld::launch_verify(a, stream);
    if (e != hipSuccess)
        return hip_fail(e, "verification launch");
    return PLD_OK;
}

pld_status pld_kv_append_tree(pld_ctx *ctx, const void *q, int64_t q_stride, const void *k,
                              const void *v, int64_t kv_stride, int32_t rows,
                              const int32_t *lengths, const int32_t *draft_len,
                              const int32_t *parent, int32_t batch, const int32_t *page_table,
                              int64_t table_stride, void *k_cache, void *v_cache,
                              int64_t n_pages, const float *k_scale, const float *v_scale,
                              const float *q_norm, const float *k_norm, float eps, void *out_q,
                              hipStream_t stream)
{
    pld::TreeAppendArgs a;
    pld_status st =
        append_args(ctx, q, q_stride, k, v, kv_stride, rows, lengths, draft_len, batch, page_table,
                    table_stride, k_cache, v_cache, n_pages, k_scale, v_scale, out_q, a.kv);
    if (st == PLD_OK && parent)
        st = tree_rows(rows, parent);
    if (st != PLD_OK)
        return st;
    if (((uintptr_t)q_norm | (uintptr_t)k_norm) & 3u)
        return fail(PLD_EINVAL, "q_norm and k_norm must be 4-byte aligned");
    if (q_norm && !q && batch > 0)
        return fail(PLD_EINVAL, "q_norm needs q");
    if (!(eps >= 0.0f) || !isfinite(eps))
        return fail(PLD_EINVAL, "eps must be >= 0 and finite");
    if (batch == 0)
        return PLD_OK;
    a.parent = parent;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    const hipError_t e = pld::launch_kv_append_tree(a, stream);
    if (e != hipSuccess)
        return hip_fail(e, "cache append launch");
    return PLD_OK;
}

pld_status pld_attend_tree(pld_ctx *ctx, const void *q, int64_t q_stride, int32_t rows,
                           const int32_t *lengths, const int32_t *draft_len,
                           const int32_t *parent, int64_t max_len, int32_t batch,
                           const int32_t *page_table, int64_t table_stride, const void *k_cache,
                           const void *v_cache, int64_t n_pages, const float *k_scale,
                           const float *v_scale, float scale, int32_t window, void *out,
                           float *out_lse, hipStream_t stream)
{
    pld::AttendArgs a;
    pld_status st =
        attend_args(ctx, q, q_stride, rows, lengths, draft_len, max_len, batch, page_table,
                    table_stride, k_cache, v_cache, n_pages, k_scale, v_scale, scale, window, out,
                    out_lse, a);
    if (st == PLD_OK && parent)
        st = tree_rows(rows, parent);
    if (st != PLD_OK || batch == 0)
        return st;
    a.parent = parent;
    // (one row is a chain)
    const hipError_t e = parent && rows > 1 ? pld::launch_attend_tree(a, stream)
                                            : pld::launch_attend(a, stream);
    if (e != hipSuccess)
        return hip_fail(e, "attention launch");
    return PLD_OK;
}

pld_status pld_verify_tree(pld_ctx *ctx, const void *logits, int32_t logits_dtype,
                           int64_t logits_stride, int32_t rows, const int32_t *draft,
                           const int32_t *draft_len, const int32_t *parent,
                           const float *temperature, const float *uniform, int32_t batch,
                           int32_t *out_tokens, int32_t *out_path, int32_t *out_accepted,
                           int32_t *out_counts, float *out_logprobs, hipStream_t stream)
{
    pld::TreeVerifyArgs a;
    pld_status st =
        verify_args(ctx, logits, logits_dtype, logits_stride, rows, draft, draft_len, nullptr,
                    nullptr, 0, temperature, uniform, batch, out_tokens, out_accepted, out_counts,
                    out_logprobs, a.v);
    if (st == PLD_OK)
        st = tree_rows(rows, parent);
    if (st != PLD_OK)
        return st;
    if (batch > 0 && !out_path)
        return fail(PLD_EINVAL, "null buffer pointer");
    if ((uintptr_t)out_path & 3u)
        return fail(PLD_EINVAL, "out_path must be 4-byte aligned");
    if (batch == 0)
        return PLD_OK;
    a.parent = parent;
    a.out_path = out_path;
    const hipError_t e = pld::launch_verify_tree(a, stream);
    if (e != hipSuccess)
        return hip_fail(e, "verification launch");
    return PLD_OK;
}

pld_status pld_kv_keep(pld_ctx *ctx, const int32_t *lengths, const int32_t *draft_len,
                       const int32_t *path, const int32_t *accepted, int32_t rows, int32_t batch,
                       const int32_t *page_table, int64_t table_stride, void *k_cache,
                       void *v_cache, int64_t n_pages, int32_t layers, int64_t k_layer_stride,
                       int64_t v_layer_stride, hipStream_t stream)
{
    pld::KeepArgs a;
    pld_status st = block_args(ctx, rows, lengths, draft_len, 0, batch, page_table, table_stride,
                               k_cache, v_cache, n_pages, nullptr, nullptr, a.blk);
    if (st == PLD_OK)
        st = tree_rows(rows, nullptr);
    if (st != PLD_OK)
        return st;
    if (batch > 0 && (!path || !accepted))
        return fail(PLD_EINVAL, "null buffer pointer");
    if (((uintptr_t)path | (uintptr_t)accepted) & 3u)
        return fail(PLD_EINVAL, "int32 and float buffers must be 4-byte aligned");
    if (layers < 0)
        return fail(PLD_EINVAL, "layers must be >= 0 (got %d)", layers);
    if (layers > 1) {
        // (2^31 pages, 2^16 heads, 2^8 positions and dims: below 2^63)
        const int64_t cells = n_pages * a.blk.kv_heads * ctx->target->p.page_tokens *
                              (int64_t)a.blk.head_dim;
        const int64_t word = a.blk.cache_dtype == PLD_E4M3 ? 16 : 8;
        if (k_layer_stride < cells || v_layer_stride < cells || k_layer_stride % word ||
            v_layer_stride % word)
            return fail(PLD_EINVAL, "k_layer_stride and v_layer_stride must hold a layer's cache "
                        "(%lld elements) and be multiples of 16 bytes", (long long)cells);
    }
    if (batch == 0 || layers == 0)
        return PLD_OK;
    a.path = path;
    a.accepted = accepted;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.layers = layers;
    a.k_layer = layers > 1 ? k_layer_stride : 0;
    a.v_layer = layers > 1 ? v_layer_stride : 0;
    const hipError_t e = pld::launch_kv_keep(a, stream);
    if (e != hipSuccess)
        return hip_fail(e, "kept cells launch");
    return PLD_OK;
}

}  // extern "C"
