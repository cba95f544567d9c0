// A tree as a wavefront holds it: lane l has the parents of nodes l, 64 + l, ...
#pragma once

#include <hip/hip_runtime.h>

#include "pld_tree.h"

namespace pld {

struct WaveTree {
    static constexpr int kParts = kTreeRows / 64;
    int32_t up[kParts];  // 0 for the root and for what is no node

    // Reads request b's tree; true where a parent is not a node before its
    // child (nothing may follow the parents then).
    __device__ __forceinline__ bool load(const int32_t *parent, const BlockArgs &g, int32_t b,
                                         int lane)
    {
        bool stray = false;
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            up[i] = parent_of(parent, g, b, i * 64 + lane, stray);
        return __any(stray);
    }

    // Steps from node t, the same on every lane, up to the root. Parents come
    // before their children, so a part is left for good.
    __device__ __forceinline__ int32_t depth(int32_t t) const
    {
        int32_t at = __builtin_amdgcn_readfirstlane(t), steps = 0;
#pragma unroll
        for (int i = kParts - 1; i >= 0; --i)
            for (; at > 0 && at >= i * 64; ++steps)
                at = __builtin_amdgcn_readlane(up[i], at - i * 64);
        return steps;
    }
};

}  // namespace pld
