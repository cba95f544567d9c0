// The context behind pld_ctx and the error report of the C-ABI layer,
// shared by its source files. Not installed; callers use include/pld.h.
#ifndef PLD_CTX_H_
#define PLD_CTX_H_

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "pld.h"
#include "pld_kernels.h"

namespace pld {

struct Target;

// Record a failure's text for pld_last_error and return its status.
pld_status fail(pld_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
pld_status hip_fail(hipError_t e, const char *what);

}  // namespace pld

struct pld_ctx {
    int device;
    int32_t max_batch;
    int32_t max_len;
    int32_t tile_tokens;        // scan tile size; 0: chosen per call (pick_tile)
    int32_t fused;
    pld::ReqSlot *slots;        // [max_batch] reduction state
    unsigned int *err;          // one word
    int4 *zero16;               // 16 zero bytes
    int32_t *store;             // [max_batch * pitch] or null
    int64_t pitch;              // tokens per store row
    int32_t *store_len;         // [max_batch] or null
    const int32_t **store_rows; // [max_batch] device row pointers or null
    unsigned long long *index;  // n-gram index over the store, or null
    int64_t index_cap;          // slots per (request, length) table
    int32_t index_lo, index_hi; // indexed lengths
    int32_t index_chunks;       // workgroups per request for an append's inserts
    uint32_t index_fp_mask;     // fingerprint bits kept
    unsigned long long *ngram_grams;  // successor-count cache: gram slots, or null
    unsigned long long *ngram_pairs;  // and pair slots
    int64_t ngram_cap;                // slots per (request, length) table
    int32_t ngram_n_max;              // context lengths 1..ngram_n_max
    int32_t ngram_chunks;             // workgroups per request for a large append
    pld::Target *target;              // the verify step's state, or null
};

#endif  // PLD_CTX_H_
