// pld_verify_tree's kernels on the host (see hip/hip_runtime.h): one call, over
// a workspace that the caller keeps between calls.
#include <hip/hip_runtime.h>

#define __builtin_amdgcn_readlane(x, i) host_device::from_lane(x, (i) & 63)
// (a workgroup runs alone: what it would wait for must not be left to others)
#define __builtin_amdgcn_s_sleep(n) abort()

#include "pld_tree_verify.hip"

extern "C" {

// order: the wavefronts' order; report: broken barriers, stuck workgroups. walk:
// only the rows on the path are read, whatever the sizes, in pieces of 2,048
// logits.
int host_verify_tree(const pld::TreeVerifyArgs *a, const int32_t *order, int32_t waves,
                     int32_t walk, int64_t *report)
{
    host_device::State &s = host_device::state();
    s.order.assign(order, order + waves);
    s.broken_barriers = s.stuck = 0;
    hipError_t e;
    if (walk) {
        const pld::VerifyArgs &v = a->v;
        const pld::Space sp =
            pld::space_of((char *)v.stats, v.max_batch, v.max_rows, v.vocab, nullptr);
        const int64_t pieces = pld::pieces_of(v.vocab, pld::kMinPiece);
        const auto both = [&](auto x, auto words) {
            typedef decltype(x) T;
            const hipError_t w = pld::launch_walk<T, words.value>(*a, sp, pieces, nullptr);
            return w != hipSuccess ? w : pld::launch_draw<T, 8>(*a, sp, nullptr);
        };
        e = v.dtype == PLD_F32
                ? both(0.0f, std::integral_constant<int, 2>())
                : (v.dtype == PLD_F16 ? both((_Float16)0, std::integral_constant<int, 1>())
                                      : both((__bf16)0, std::integral_constant<int, 1>()));
    } else {
        e = pld::launch_verify_tree(*a, nullptr);
    }
    report[0] = s.broken_barriers;
    report[1] = s.stuck;
    return e;
}

// The launches of a call of these sizes, not run: the threads of the largest
// grid, or 0 where the sizes are refused.
uint64_t host_verify_tree_grid(int32_t batch, int32_t rows, int32_t vocab, int32_t dtype)
{
    pld::TreeVerifyArgs a;
    memset(&a, 0, sizeof(a));
    a.v.dtype = dtype;
    a.v.rows = a.v.max_rows = rows;
    a.v.batch = a.v.max_batch = batch;
    a.v.vocab = vocab;
    host_device::State &s = host_device::state();
    s.dry = true;
    s.most_threads = 0;
    const hipError_t e = pld::launch_verify_tree(a, nullptr);
    s.dry = false;
    return e == hipSuccess ? s.most_threads : 0;
}

}
