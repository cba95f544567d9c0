// The tree that a request's drafted tokens form: its parents are checked here
// before anything follows them. Plain C++ but for the walk that a wavefront
// does, so that a host test can run it.
#pragma once

#include <stdint.h>

#include "pld_block.h"
#include "pld_target.h"

namespace pld {

// Nodes of a tree, its root included: PLD_TREE_ROWS.
constexpr int32_t kTreeRows = PLD_TREE_ROWS;

// The parent of request b's node t: 0 for the root and for what is no node of
// the tree; `stray` is set where it is not a node before t.
PLD_INLINE int32_t parent_of(const int32_t *parent, const BlockArgs &g, int32_t b, int32_t t,
                             bool &stray)
{
    // (a draft length past the block is refused elsewhere: nothing is read for it)
    if (t < 1 || t >= g.rows || t > g.draft_len[b])
        return 0;
    const int32_t p = parent ? parent[(int64_t)b * (g.rows - 1) + t - 1] : t - 1;
    if (p >= 0 && p < t)
        return p;
    stray = true;
    return 0;
}

}  // namespace pld
