// Attention of a tree's rows over the paged cache, for gfx950 (MI355X): the
// kernels of pld_attend_device.h for blocks that are trees.

#include "pld_attend_device.h"

namespace pld {

hipError_t launch_attend_tree(const AttendArgs &a, hipStream_t s)
{
    return launch_blocks<true>(a, s);
}

}  // namespace pld
