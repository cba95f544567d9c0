// Attention of the verify block's rows over the paged cache, for gfx950
// (MI355X): the kernels of pld_attend_device.h for blocks that are chains.

#include "pld_attend_launch.h"

namespace pld {

// Enough for kMostGroups workgroups of 64 rows, or for every span of the
// shortest kind that the context's calls can have.
int64_t attend_rows(const pld_target_params &p)
{
    const int64_t group = p.q_heads / p.kv_heads;
    const int64_t rows = (p.max_rows * group + 127) / 128 * 128 * p.max_batch * p.kv_heads;
    const int64_t spans = ceil_div(p.max_len, kMinSpan);
    const int64_t most = 64 * kMostGroups;
    return spans >= ceil_div(most, rows) ? most : rows * spans;
}

hipError_t launch_attend(const AttendArgs &a, hipStream_t s)
{
    return a.blk.dtype == PLD_BF16 ? launch_blocks<__bf16, false>(a, s)
                                   : launch_blocks<_Float16, false>(a, s);
}

}  // namespace pld
