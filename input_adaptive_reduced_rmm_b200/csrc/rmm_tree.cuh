// rmm_tree.cuh -- the draft tree as the kernels read it.
//
// A tree of up to 64 nodes is an int32 array of parents, parent before child:
// parents[t] in [0, t) hangs node t on that node, -1 makes it a root, anything
// else marks it absent (padding).  A node below an absent one is absent too.
#pragma once

#include <stdint.h>

namespace rmm {

constexpr int kTreeMax = 64;        // nodes per tree: a node's way to its root is one 64-bit word
constexpr int kTreeMaxBatch = 4096; // sequences per call
constexpr int kTreeMaxHeads = 4096; // heads of a kind

// Node t and its ancestors as a bit mask, 0 when t is absent.  Parents are
// strictly smaller than their children, so the walk ends after at most t steps
// whatever the array holds.
__device__ __forceinline__ uint64_t tree_way(const int32_t* parents, int t) {
    uint64_t way = 0;
    for (int n = t;;) {
        way |= 1ull << n;
        const int p = parents[n];
        if (p == -1) return way;
        if (p < 0 || p >= n) return 0;
        n = p;
    }
}

// The same for a chain (no tree given): node t sees nodes 0 .. t.
__device__ __forceinline__ uint64_t chain_way(int t) { return ~0ull >> (63 - t); }

}  // namespace rmm
