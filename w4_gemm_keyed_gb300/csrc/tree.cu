// Acceptance along trees of drafted tokens, and the cache entries of the accepted
// paths.
#include "tree.cuh"

namespace tfk {

namespace {

// ------------------------------------------------------------- acceptance
// A warp per sequence, two nodes a lane.  Each step asks every node at once whether
// it is a child of the walk's last node that holds the token sampled there; the
// first that answers goes on.  At most kMaxPath steps of a ballot each: the launch
// bounds it (64 sequences of 64 nodes 4 us).
constexpr int kAcceptWarps = 4;

__global__ void __launch_bounds__(32 * kAcceptWarps) tree_accept_kernel(TreeAcceptArgs a) {
    grid_dependency_wait();     // the sampled tokens come from the preceding grid
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, b = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5), n = a.n;
    if (b >= a.n_seq) return;
    const long long pos = a.pos[b];
    const size_t row = (size_t)b * n;
    int d[2], parent[2], token[2], sampled[2];
    bool go = tree_depths(a.parents + row, n, d);
    if (lane == 0 && pos >= 0 && !go) set_error(a.err, kDevBadTree);
    if (lane == 0 && pos < -1) set_error(a.err, kDevBadPosition);
    go = go && pos >= 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        const bool used = i < n && d[h] > 0;
        parent[h] = used ? a.parents[row + i] : -1;
        token[h] = used ? a.tokens[row + i] : 0;
        sampled[h] = i < n ? a.sampled[row + i] : 0;
    }
    int at = 0, steps = -1, my_node = -1, my_token = -1, last = -1;
    while (go) {
        const int s0 = __shfl_sync(0xFFFFFFFFu, sampled[0], at & 31), s1 = __shfl_sync(0xFFFFFFFFu, sampled[1], at & 31);
        last = at < 32 ? s0 : s1;
        ++steps;
        if (lane == steps) {
            my_node = at;
            my_token = last;
        }
        const unsigned lo = __ballot_sync(0xFFFFFFFFu, parent[0] == at && token[0] == last);
        const unsigned hi = __ballot_sync(0xFFFFFFFFu, parent[1] == at && token[1] == last);
        go = (lo | hi) != 0u;
        if (go) at = lo ? __ffs(lo) - 1 : __ffs(hi) + 31;       // a child's number is above its parent's: this ends
    }
    if (lane < kMaxPath) {
        a.path[(size_t)b * kMaxPath + lane] = my_node;
        a.committed[(size_t)b * kMaxPath + lane] = my_token;
    }
    if (lane == 0) {
        a.accepted[b] = steps;
        a.bonus[b] = last;
    }
}

// ------------------------------------------------------- an accepted path's entries
// A node's number is at least its depth, so entries move towards the front; a warp
// takes all depths of one (sequence, head, K or V) vector by vector's 16-byte chunk:
// lanes 0-15 one chunk of depth d, lanes 16-31 of depth d + 1, all loads before the
// first store.  A path must rise strictly from node 0.  The launch and three loads in a row bound it (64 sequences,
// 8 heads, E4M3, 4 us).
constexpr int kKeepWarps = 4;

template <bool E4M3>
__global__ void __launch_bounds__(32 * kKeepWarps) kv_keep_kernel(KvBatch c, const int64_t *pos, const int32_t *path,
                                                                  int *err) {
    grid_dependency_wait();     // the path comes from the preceding grid
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, unit = blockIdx.x * kKeepWarps + (threadIdx.x >> 5), b = blockIdx.y;
    if (unit >= 2 * c.n_kv) return;
    const long long p = pos[b];
    const int node = lane < kMaxPath ? path[(size_t)b * kMaxPath + lane] : -1;
    const int before = __shfl_up_sync(0xFFFFFFFFu, node, 1);
    const unsigned used = __ballot_sync(0xFFFFFFFFu, node >= 0);
    const int n = __popc(used);
    // -1 marks the rows after the path's end; the path starts at node 0 and rises
    bool bad = node < -1 || node >= kMaxNodes || (used & (used + 1u)) != 0u ||
               (node >= 0 && (lane == 0 ? node != 0 : node <= before));
    const int last = __shfl_sync(0xFFFFFFFFu, node, max(n, 1) - 1);
    bad = __any_sync(0xFFFFFFFFu, bad);
    // no sum with p: it may be any int64
    const bool out = p < -1 || p > (long long)c.max_len - 1 - last;
    if (p != -1 && (bad || out) && unit == 0 && lane == 0) set_error(err, out ? kDevBadPosition : kDevBadTree);
    if (p < 0 || bad || out || n < 2) return;
    const int j = unit >> 1;
    const size_t base = (size_t)(b * c.n_kv + j) * c.max_len + (size_t)p;
    constexpr int kBytes = E4M3 ? kHeadDim : 2 * kHeadDim, kLanes = kBytes / 16;    // lanes of a vector
    constexpr int kAtOnce = 32 / kLanes, kSteps = kMaxPath / kAtOnce;
    uint8_t *const data = static_cast<uint8_t *>(unit & 1 ? c.v : c.k);
    uint8_t *const scale = unit & 1 ? c.v_scale : c.k_scale;
    uint4 x[kSteps];
    const int chunk = lane % kLanes, sub = lane / kLanes;
    auto at = [&](size_t entry) {       // bf16: chunks are permuted by position, max_len % 8 = 0
        return reinterpret_cast<uint4 *>(data + entry * kBytes + 16 * (E4M3 ? chunk : chunk ^ int(entry & 7)));
    };
    int s = 0;
    if (E4M3 && lane < n) s = scale[base + node];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int d = i * kAtOnce + sub, from = __shfl_sync(0xFFFFFFFFu, node, d);
        if (d < n) x[i] = *at(base + from);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int d = i * kAtOnce + sub;
        if (d < n) *at(base + d) = x[i];
    }
    if (E4M3 && lane < n) scale[base + lane] = uint8_t(s);
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptArgs &a, cudaStream_t s) {
    return launch_pdl(tree_accept_kernel, dim3((a.n_seq + kAcceptWarps - 1) / kAcceptWarps), dim3(32 * kAcceptWarps), 0, s, a);
}

cudaError_t launch_kv_keep(const KvBatch &c, const int64_t *pos, const int32_t *path, int *err, cudaStream_t s) {
    const dim3 grid((2 * c.n_kv + kKeepWarps - 1) / kKeepWarps, c.n_seq), block(32 * kKeepWarps);
    return c.format == kKvE4m3 ? launch_pdl(kv_keep_kernel<true>, grid, block, 0, s, c, pos, path, err)
                               : launch_pdl(kv_keep_kernel<false>, grid, block, 0, s, c, pos, path, err);
}

}  // namespace tfk
