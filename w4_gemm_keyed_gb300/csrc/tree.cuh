// Trees of drafted tokens: their shape, acceptance along them, and the entries of an
// accepted path.
#pragma once
#include "kv_batch.cuh"

namespace tfk {

constexpr int kMaxNodes = 64;       // nodes of a tree, unused rows included
constexpr int kMaxPath = 16;        // nodes on a path, the root included
constexpr int kDevBadTree = 5;      // device status: parents or a path that no tree has

// Depths of a tree's nodes: d[h] is node lane + 32 h's, -1 for an unused row.  Whole
// converged warp; parents: the sequence's n entries.  False (in all lanes) where the parents are no tree:
// parents[0] must be -1, a used node's parent a used node before it, and no path
// longer than kMaxPath.  Depths by doubling: after r rounds `up` is the ancestor
// 2^r steps up (the root where there are fewer) and d counts the steps.
__device__ __forceinline__ bool tree_depths(const int32_t *parents, int n, int (&d)[2]) {
    const int lane = threadIdx.x & 31;
    int up[2];
    bool bad = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        const int p = i < n ? parents[i] : -1;
        bad |= p >= i || p < -1;        // node 0: anything but -1
        d[h] = i == 0 ? 0 : (p < 0 ? -1 : 1);
        up[h] = p < 0 || p >= i ? 0 : p;
    }
    auto of = [](const int (&v)[2], int i) {
        const int a = __shfl_sync(0xFFFFFFFFu, v[0], i & 31), b = __shfl_sync(0xFFFFFFFFu, v[1], i & 31);
        return i < 32 ? a : b;
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int p = of(d, up[h]);
        bad |= d[h] > 0 && p < 0;       // the parent is unused
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int e0 = of(d, up[0]), e1 = of(d, up[1]), u0 = of(up, up[0]), u1 = of(up, up[1]);
        if (d[0] > 0) d[0] += e0;
        if (d[1] > 0) d[1] += e1;
        up[0] = u0;
        up[1] = u1;
    }
    // 16 steps up is past the root of every path that is short enough
    bad |= up[0] != 0 || up[1] != 0 || d[0] >= kMaxPath || d[1] >= kMaxPath;
    return !__any_sync(0xFFFFFFFFu, bad);
}

struct TreeAcceptArgs {
    const int32_t *parents, *tokens, *sampled;  // [n_seq][n]
    const int64_t *pos;                         // [n_seq]
    int n_seq, n;
    int32_t *accepted, *bonus;                  // [n_seq]
    int32_t *path, *committed;                  // [n_seq][kMaxPath]
    int *err;
};
cudaError_t launch_tree_accept(const TreeAcceptArgs &a, cudaStream_t s);

// entries pos[b] + path[b][d] -> pos[b] + d
cudaError_t launch_kv_keep(const KvBatch &c, const int64_t *pos, const int32_t *path, int *err, cudaStream_t s);

}  // namespace tfk
