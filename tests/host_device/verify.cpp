// pld_verify's kernels on the host (see hip/hip_runtime.h): one call, over a
// workspace that the caller keeps between calls.
#include "pld_verify.hip"

extern "C" {

size_t host_workspace(int32_t batch, int32_t rows, int32_t vocab)
{
    return pld::verify_workspace(batch, rows, vocab);
}

int host_clear(void *ws, int32_t batch, int32_t rows, int32_t vocab)
{
    return pld::verify_clear(ws, batch, rows, vocab, nullptr);
}

// Whether the counters are as a call must leave them.
int host_counters_clear(void *ws, int32_t batch, int32_t rows, int32_t vocab)
{
    const pld::Space sp = pld::space_of((char *)ws, batch, rows, vocab, nullptr);
    for (int64_t i = 0; i < (int64_t)batch * rows; ++i)
        if (sp.arrived[i])
            return 0;
    for (int32_t b = 0; b < batch; ++b)
        if (sp.drawn[b] || sp.stop[b] != pld::kNever)
            return 0;
    return 1;
}

// The launches of a call of these sizes, not run: the threads of the largest
// grid, or 0 where the sizes are refused.
uint64_t host_verify_grid(int32_t batch, int32_t rows, int32_t vocab, int32_t dtype, int32_t head)
{
    pld::VerifyArgs a;
    memset(&a, 0, sizeof(a));
    a.dtype = dtype;
    a.rows = a.max_rows = rows;
    a.batch = a.max_batch = batch;
    a.vocab = vocab;
    a.head = head;
    host_device::State &s = host_device::state();
    s.dry = true;
    s.most_threads = 0;
    const hipError_t e = pld::launch_verify(a, nullptr);
    s.dry = false;
    return e == hipSuccess ? s.most_threads : 0;
}

// order: the wavefronts' order, `waves` of them. refuse_row > 0: `refuse_row`
// is refused by another workgroup between the looks that two wavefronts of a
// workgroup take at `stop`: the first finds no refusal, the others find it.
// report: broken barriers, stuck workgroups.
int host_verify(const pld::VerifyArgs *a, const int32_t *order, int32_t waves, int32_t refuse_row,
                int64_t *report)
{
    host_device::State &s = host_device::state();
    s.order.assign(order, order + waves);
    s.broken_barriers = s.stuck = 0;
    s.on_load = nullptr;
    const pld::Space sp = pld::space_of((char *)a->stats, a->max_batch, a->max_rows, a->vocab,
                                        nullptr);
    uint32_t looked_block = ~0u, looked_wave = 0;
    if (refuse_row > 0)
        s.on_load = [&](const void *p) {
            int32_t *word = (int32_t *)p;
            if (word < sp.stop || word >= sp.stop + a->max_batch)
                return;
            if (looked_block != blockIdx.x) {
                looked_block = blockIdx.x;
                looked_wave = threadIdx.x / 64;
            }
            *word = threadIdx.x / 64 == looked_wave ? pld::kNever : refuse_row;
        };
    const hipError_t e = pld::launch_verify(*a, nullptr);
    s.on_load = nullptr;
    report[0] = s.broken_barriers;
    report[1] = s.stuck;
    return e;
}

}
