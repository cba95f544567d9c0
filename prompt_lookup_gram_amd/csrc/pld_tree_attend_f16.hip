// Attention of a tree's rows over the paged cache, for gfx950 (MI355X): the
// kernels of pld_tree_attend.hip in f16.

#include "pld_attend_launch.h"

namespace pld {

hipError_t launch_attend_tree_f16(const AttendArgs &a, hipStream_t s)
{
    return launch_blocks<_Float16, true>(a, s);
}

}  // namespace pld
