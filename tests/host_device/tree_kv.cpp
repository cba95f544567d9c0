// pld_kv_append_tree's and pld_kv_keep's kernels on the host (see
// hip/hip_runtime.h).
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

#include <hip/hip_runtime.h>

#define __builtin_amdgcn_readlane(x, i) host_device::from_lane(x, (i) & 63)
#define __builtin_amdgcn_wave_barrier() ((void)host_device::exchange(0))
#define __builtin_amdgcn_fence(order, scope) ((void)0)

#include "pld_tree_kv.hip"

extern "C" {

// order: the wavefronts' order; report: broken barriers, stuck workgroups.
int host_append_tree(const pld::TreeAppendArgs *a, const int32_t *order, int32_t waves,
                     int64_t *report)
{
    host_device::State &s = host_device::state();
    s.order.assign(order, order + waves);
    s.broken_barriers = s.stuck = 0;
    const hipError_t e = pld::launch_kv_append_tree(*a, nullptr);
    report[0] = s.broken_barriers;
    report[1] = s.stuck;
    return e;
}

int host_kv_keep(const pld::KeepArgs *a, const int32_t *order, int32_t waves, int64_t *report)
{
    host_device::State &s = host_device::state();
    s.order.assign(order, order + waves);
    s.broken_barriers = s.stuck = 0;
    const hipError_t e = pld::launch_kv_keep(*a, nullptr);
    report[0] = s.broken_barriers;
    report[1] = s.stuck;
    return e;
}

}
