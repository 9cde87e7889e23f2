// The contract's tile tree as threads evaluate it: which tiles a thread merges
// in its registers, and the levels across lanes (rlk_merge.cu says how the
// tree is laid over threads).  Shared by the tile-tree kernels and the draft
// verification.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "rlk_contract.cuh"

namespace rlk {

// The slots a thread owns form one node of the perfect tree; its tiles are a
// contiguous run (the bisection keeps tile order): `first` tile, `count` tiles.
struct SlotRun {
    int first;
    int count;
};

// Node of thread u when a token's 2^max(depth, log2 P) slots are spread over
// P = 2^kLogP threads.  The contract's tree occupies the first 2^depth slots;
// walking its bisection down u's bits (most significant first) gives the
// node.  With fewer slots than threads, thread u holds slot u alone.
template <int kLogP>
__device__ __forceinline__ SlotRun slot_run(int u, int depth, int n_tiles) {
    SlotRun r;
    r.first = 0;
    r.count = n_tiles;
    int levels = kLogP;
    if (depth < kLogP) {
        if (u >= (1 << depth)) {
            r.count = 0;
            return r;
        }
        levels = depth;
    }
    for (int b = levels - 1; b >= 0; --b) {
        const int left = (r.count + 1) >> 1;
        if ((u >> b) & 1) {
            r.first += left;
            r.count -= left;
        } else {
            r.count = left;
        }
    }
    return r;
}

// Merge a thread's node of one token's tree: its L = 2^kLogL slots of the
// perfect tree (levels 1 .. kLogL).  In a bisection of k tiles over 2^h
// slots (larger half first), slot j holds a tile exactly when the h-bit
// reversal of j is below k, and the tiles fill the held slots in order.  A
// thread's node holds between L/2 and L tiles (bisection keeps the nodes of
// one depth within one tile of each other, and the tree has 2^depth slots
// for at most 2^depth and more than 2^(depth-1) tiles), so every even slot
// 2i holds a tile (its reversal is that of i, below L/2), and the odd slot
// 2i+1 holds one exactly when the (h-1)-bit reversal of i is below k - L/2.
// Level 1 therefore merges a pair only where the odd slot is held -- a
// lone even slot is its own level-1 node, as in the bisection tree, whose
// nodes never see an empty operand -- and levels 2 .. kLogL, over nodes that
// all hold tiles, run as a binary counter (a node is formed as soon as both
// children exist).  load(k) returns tile k's (max, sum) pair; `present`
// says whether the node holds any tile (only L = 1 nodes can be empty).
template <int kLogL, typename Load>
__device__ __forceinline__ MaxSum merge_run(const SlotRun& run, Load load, bool& present) {
    MaxSum x;
    if constexpr (kLogL == 0) {
        present = run.count > 0;
        x.m = -CUDART_INF_F;
        x.s = 0.0f;
        if (present) {
            const float2 p = load(run.first);
            x.m = p.x;
            x.s = p.y;
        }
    } else {
        constexpr int kPairs = 1 << (kLogL - 1);
        const int odd_limit = run.count - kPairs;
        MaxSum pend[kLogL];
        int rel = 0;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const float2 p = load(run.first + rel);
            ++rel;
            x.m = p.x;
            x.s = p.y;
            const int rev =
                kLogL > 1 ? static_cast<int>(__brev(static_cast<unsigned>(i)) >> (33 - kLogL)) : 0;
            if (rev < odd_limit) {
                const float2 q = load(run.first + rel);
                ++rel;
                MaxSum y;
                y.m = q.x;
                y.s = q.y;
                x = contract_merge(x, y);
            }
            int level = 0;
#pragma unroll
            for (; level < kLogL - 1; ++level) {
                if (!(i & (1 << level))) break;
                x = contract_merge(pend[level], x);  // left sibling + this node
            }
            if (level < kLogL - 1) pend[level] = x;
        }
        present = true;
    }
    return x;
}

// One merge level across lanes: partner lane ^ (1 << lv), the lower lane
// left; a side without tiles leaves the other unchanged.
__device__ __forceinline__ MaxSum shuffle_level(MaxSum x, bool& xp, int lane, int lv) {
    MaxSum o;
    o.m = __shfl_xor_sync(0xffffffffu, x.m, 1 << lv);
    o.s = __shfl_xor_sync(0xffffffffu, x.s, 1 << lv);
    const bool op = __shfl_xor_sync(0xffffffffu, xp ? 1 : 0, 1 << lv) != 0;
    MaxSum r = x;
    if (xp && op) r = (lane & (1 << lv)) ? contract_merge(o, x) : contract_merge(x, o);
    else if (op) r = o;
    xp = xp || op;
    return r;
}

}  // namespace rlk
