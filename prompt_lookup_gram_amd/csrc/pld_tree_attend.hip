// Attention of a tree's rows over the paged cache, for gfx950 (MI355X): the
// kernels of pld_attend_device.h and pld_attend_tall.h for blocks that are trees,
// in bf16. (f16 is a source of its own: each takes the compiler minutes.)

#include "pld_attend_launch.h"

namespace pld {

hipError_t launch_attend_tree(const AttendArgs &a, hipStream_t s)
{
    return a.blk.dtype == PLD_BF16 ? launch_blocks<__bf16, true>(a, s)
                                   : launch_attend_tree_f16(a, s);
}

}  // namespace pld
