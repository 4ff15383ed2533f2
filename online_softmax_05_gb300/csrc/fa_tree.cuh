// fa_tree.cuh -- the tree of a sequence's drafted tokens, from the places' parents.
#pragma once

#include <cuda_runtime.h>

namespace fa {

constexpr int kTreePlaces = 64;  // most places of a tree

// A warp finds, for the places lane and lane + 32, the places from the root to each of them
// (bit i: place i, itself among them); 0 where parents[] leads to no root or i is at or
// behind N.  A parent is -1 (a root) or below its place.  Each round the paths
// known so far double: six for 64 places.
__device__ __forceinline__ void tree_ancestors(const int* parents, int N, int lane, unsigned long long (&up)[2]) {
    int at[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x;
        at[x] = i < N ? __ldg(parents + i) : -2;
        if (at[x] < -1 || at[x] >= i) at[x] = -2;
        up[x] = 1ull << i | (at[x] >= 0 ? 1ull << at[x] : 0ull);
    }
#pragma unroll
    for (int round = 0; round < 6; ++round) {
        unsigned long long more[2];
        int to[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int src = at[x] & 31;
            const unsigned long long a = __shfl_sync(0xffffffffu, up[0], src), b = __shfl_sync(0xffffffffu, up[1], src);
            const int c = __shfl_sync(0xffffffffu, at[0], src), d = __shfl_sync(0xffffffffu, at[1], src);
            const bool going = at[x] >= 0, high = at[x] >= 32;
            more[x] = going ? (high ? b : a) : 0ull;
            to[x] = going ? (high ? d : c) : at[x];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            up[x] |= more[x];
            at[x] = to[x];
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
        if (at[x] != -1) up[x] = 0;
}

}  // namespace fa
