// Internal interface of the verify step's operators: the state a target
// context holds, the kernels' arguments and their launches. Not installed;
// callers use include/pld.h.
#ifndef PLD_TARGET_H_
#define PLD_TARGET_H_

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "pld.h"

namespace pld {

// A batch's blocks and the paged cache they stand in.
struct BlockArgs {
    const int32_t *lengths;    // [batch]
    const int32_t *draft_len;  // [batch]
    int32_t rows;              // rows of a padded block
    int32_t batch;
    int32_t max_len;           // bound on lengths[b] + draft_len[b]
    const int32_t *table;
    int64_t table_stride;
    int64_t n_pages;
    int32_t page_shift;        // log2 of page_tokens
    int32_t q_heads, kv_heads, head_dim;
    int32_t dtype, cache_dtype;
    const float *k_scale;      // [kv_heads] or null
    const float *v_scale;
    unsigned int *err;
};

struct KvAppendArgs {
    BlockArgs blk;
    const void *q;             // or null
    int64_t q_stride;
    const void *k;
    const void *v;
    int64_t kv_stride;
    void *k_cache;
    void *v_cache;
    void *out_q;
    const double *turns;       // [rot_dim / 2] turns per position of each pair
    int32_t rot_dim, interleaved;
    float magnitude;
};

struct AttendArgs {
    BlockArgs blk;
    const void *q;
    int64_t q_stride;
    const void *k_cache;
    const void *v_cache;
    float scale;
    int32_t window;            // 0: none
    void *out;
    float *out_lse;            // or null
    float *ws;                 // workspace: partial results of ws_rows rows
    int64_t ws_rows;           // (head_dim floats each, then two floats each)
    const int32_t *parent;     // trees: [batch][rows - 1]
};

// pld_kv_append_tree
struct TreeAppendArgs {
    KvAppendArgs kv;
    const int32_t *parent;     // [batch][rows - 1], or null: chains
    const float *q_norm;       // [head_dim], or null
    const float *k_norm;
    float eps;
};

// pld_kv_keep
struct KeepArgs {
    BlockArgs blk;
    const int32_t *path;       // [batch][rows]
    const int32_t *accepted;   // [batch]
    void *k_cache;
    void *v_cache;
    int32_t layers;
    int64_t k_layer, v_layer;  // elements between layers
};

struct VerifyArgs {
    const void *logits;
    int32_t dtype;
    int64_t stride;
    int32_t rows, batch, vocab;
    const int32_t *draft;      // [batch][rows - 1]
    const int32_t *draft_len;
    const uint64_t *src;       // or null
    const float *probs;        // [batch][head][vocab] or null
    int32_t head;
    const float *temperature;  // or null
    const float *uniform;      // [batch][rows]
    int32_t *out_tokens;
    int32_t *out_accepted;
    int32_t *out_counts;
    float *out_logprobs;       // or null
    unsigned int *err;
    void *stats;               // workspace, for max_batch blocks of max_rows rows
    int32_t max_batch, max_rows;
};

// pld_verify_tree
struct TreeVerifyArgs {
    VerifyArgs v;              // (no src, probs and head)
    const int32_t *parent;     // [batch][rows - 1], or null: chains
    int32_t *out_path;         // [batch][rows]
};

// Whether one launch can have so many workgroups: the hardware counts a grid in
// threads, in 32 bits.
inline bool fits_grid(int64_t groups, int64_t threads) { return groups <= 0xffffffffLL / threads; }

// What pld_create_target adds to a context.
struct Target {
    pld_target_params p;
    int32_t page_shift;
    double *turns;       // device [rot_dim / 2]
    void *verify_ws;     // device, when vocab > 0
    float *attend_ws;    // device, when there are heads
    int64_t attend_rows;
};

void target_release(Target *t);

// Rows of partial results pld_attend's workspace should hold.
int64_t attend_rows(const pld_target_params &p);
size_t verify_workspace(int32_t batch, int32_t rows, int32_t vocab);
// Sets a new workspace's counters.
hipError_t verify_clear(void *ws, int32_t batch, int32_t rows, int32_t vocab, hipStream_t s);
hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s);
hipError_t launch_attend(const AttendArgs &a, hipStream_t s);
hipError_t launch_verify(const VerifyArgs &a, hipStream_t s);
hipError_t launch_kv_append_tree(const TreeAppendArgs &a, hipStream_t s);
hipError_t launch_attend_tree(const AttendArgs &a, hipStream_t s);
hipError_t launch_attend_tree_f16(const AttendArgs &a, hipStream_t s);
hipError_t launch_verify_tree(const TreeVerifyArgs &a, hipStream_t s);
hipError_t launch_kv_keep(const KeepArgs &a, hipStream_t s);

}  // namespace pld

#endif  // PLD_TARGET_H_
