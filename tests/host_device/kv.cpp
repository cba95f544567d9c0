// pld_kv_append's kernels on the host (see hip/hip_runtime.h).
#include <stdint.h>
#include <string.h>

// (the kernels' LDS is declared inside them, and this is it)
namespace pld {
namespace {
__attribute__((aligned(16))) char lds[160 << 10];
}
}
#define __shared__

// float to bf16, nearest even: what the compiler calls for it on the host
extern "C" __bf16 __truncsfbf2(float x)
{
    uint32_t v;
    memcpy(&v, &x, 4);
    const uint16_t r = (v & 0x7fffffffu) > 0x7f800000u ? (uint16_t)(v >> 16 | 0x40)
                                                       : (uint16_t)((v + 0x7fff + ((v >> 16) & 1)) >> 16);
    __bf16 y;
    memcpy(&y, &r, 2);
    return y;
}

#include "pld_kv.hip"

extern "C" {

// order: the wavefronts' order; report: broken barriers, stuck workgroups.
int host_kv_append(const pld::KvAppendArgs *a, const int32_t *order, int32_t waves, int64_t *report)
{
    host_device::State &s = host_device::state();
    s.order.assign(order, order + waves);
    s.broken_barriers = s.stuck = 0;
    const hipError_t e = pld::launch_kv_append(*a, nullptr);
    report[0] = s.broken_barriers;
    report[1] = s.stuck;
    return e;
}

// The launch of a call of these sizes, not run: its threads, or 0 where the
// sizes are refused. `words`: with the alignment of whole words.
uint64_t host_kv_grid(int32_t batch, int32_t rows, int32_t kv_heads, int32_t words)
{
    pld::KvAppendArgs a;
    memset(&a, 0, sizeof(a));
    a.blk.batch = batch;
    a.blk.rows = rows;
    a.blk.q_heads = a.blk.kv_heads = kv_heads;
    a.blk.head_dim = 64;
    a.blk.dtype = a.blk.cache_dtype = PLD_BF16;
    a.kv_stride = words ? 64 * kv_heads : 64 * kv_heads + 1;
    host_device::State &s = host_device::state();
    s.dry = true;
    s.most_threads = 0;
    const hipError_t e = pld::launch_kv_append(a, nullptr);
    s.dry = false;
    return e == hipSuccess ? s.most_threads : 0;
}

}
