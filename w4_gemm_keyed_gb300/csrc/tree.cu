// Acceptance along trees of drafted tokens, and the cache entries of the accepted
// paths.
#include "tree.cuh"

namespace tfk {

namespace {

constexpr float kScale = 0.08838834764831845f;      // 1 / sqrt(128)

// ------------------------------------------------------------- acceptance
// A warp per sequence, two nodes a lane.  Each step asks every node at once whether
// it is a child of the walk's last node that holds the token sampled there; the
// first that answers goes on.  At most kMaxPath steps of a ballot each: the launch
// bounds it.
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
// first store.  A path must rise strictly from node 0.
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
    const bool out = p < -1 || (p >= 0 && p + last >= c.max_len);
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

// ------------------------------------------------------- attention of a tree's nodes
// A warp per (node, query head): keys 32 at a time in the order of the path, a key per
// lane for the scores, four output columns per lane for the sums, all in fp32.
template <bool E4M3>
struct Entry {      // one half (K or V) of a cache's entries
    const void *data;
    const uint8_t *scale;
    __device__ uint32_t factor(size_t e) const { return E4M3 ? e4m3_factor(scale[e]) : 0u; }
    __device__ void eight(size_t e, int c, uint32_t f, float (&x)[8]) const {   // elements 8c .. 8c + 7
        uint32_t w[4];
        if constexpr (E4M3) {
            const uint2 p = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(data) + e * kHeadDim +
                                                             16 * (c & 7) + 8 * (c >> 3));
            e4m3_expand(p.x, f, w[0], w[1]);
            e4m3_expand(p.y, f, w[2], w[3]);
        } else {
            const uint4 p = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(data) + e * kHeadDim +
                                                             8 * (c ^ int(e & 7)));
            w[0] = p.x, w[1] = p.y, w[2] = p.z, w[3] = p.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

constexpr int kAttnWarps = 4;

template <bool E4M3>
__global__ void __launch_bounds__(32 * kAttnWarps) attn_tree_kernel(AttnTreeArgs a) {
    __shared__ float s_q[kAttnWarps][kHeadDim];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y;
    const int n_q = a.own.n_kv * a.group, unit = blockIdx.x * kAttnWarps + warp;
    if (unit >= a.n * n_q) return;
    const int node = unit / n_q, h = unit - node * n_q, j = h / a.group, row = b * a.n + node;
    const int32_t *parents = a.parents + (size_t)b * a.n;
    int d[2];
    const bool tree = tree_depths(parents, a.n, d);
    const long long pos = seq_position(a.pos, b, a.n, a.own.max_len, a.err, unit == 0 && lane == 0);
    if (unit == 0 && lane == 0 && pos >= 0 && !tree) set_error(a.err, kDevBadTree);
    const int d0 = __shfl_sync(0xFFFFFFFFu, d[0], node & 31), d1 = __shfl_sync(0xFFFFFFFFu, d[1], node & 31);
    const int depth = node < 32 ? d0 : d1;
    uint2 *out = reinterpret_cast<uint2 *>(a.out + (size_t)row * a.ldo + h * kHeadDim) + lane;
    if (pos < 0 || !tree || depth < 0) {
        *out = make_uint2(0u, 0u);
        return;
    }
    int my_node = node;     // lane t: the path's node at depth t
    for (int up = node, t = depth; t >= 0; --t, up = parents[up])
        if (lane == t) my_node = up;
    const uint16_t *q = a.q + (size_t)row * a.ldq + h * kHeadDim;
    for (int i = lane; i < kHeadDim; i += 32) s_q[warp][i] = __uint_as_float(uint32_t(q[i]) << 16) * kScale;
    __syncwarp();
    const long long total = a.prefix_len + pos + depth + 1;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (long long t0 = 0; t0 < total; t0 += 32) {
        const long long t = t0 + lane;
        const long long y = t - a.prefix_len;       // own position
        const int on = __shfl_sync(0xFFFFFFFFu, my_node, int(max(0ll, min(31ll, y - pos))));
        const bool shared = y < 0, seen = t < total;
        const Entry<E4M3> k = {shared ? a.prefix.k : a.own.k, shared ? a.prefix.k_scale : a.own.k_scale};
        const size_t e = shared ? (size_t)j * a.prefix.max_len + t
                                : (size_t)(b * a.own.n_kv + j) * a.own.max_len + (y < pos ? y : pos + on);
        float s = -INFINITY;
        if (seen) {
            s = 0.f;
            const uint32_t f = k.factor(e);
            for (int c = 0; c < 16; ++c) {
                float x[8];
                k.eight(e, c, f, x);
                for (int i = 0; i < 8; ++i) s = fmaf(x[i], s_q[warp][8 * c + i], s);
            }
        }
        float top = s;
        for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
        top = fmaxf(top, m);
        const float scale = top == -INFINITY ? 1.f : expf(m - top), w = seen ? expf(s - top) : 0.f;
        float sum = w;
        for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
        l = l * scale + sum;
        m = top;
        for (int i = 0; i < 4; ++i) o[i] *= scale;
        const int keys = int(min(32ll, total - t0));
        for (int u = 0; u < keys; ++u) {
            const float wu = __shfl_sync(0xFFFFFFFFu, w, u);
            const size_t eu = __shfl_sync(0xFFFFFFFFu, (unsigned long long)e, u);
            const bool su = t0 + u < a.prefix_len;
            const Entry<E4M3> v = {su ? a.prefix.v : a.own.v, su ? a.prefix.v_scale : a.own.v_scale};
            float x[8];
            v.eight(eu, lane >> 1, v.factor(eu), x);
            for (int i = 0; i < 4; ++i) o[i] = fmaf(wu, lane & 1 ? x[4 + i] : x[i], o[i]);
        }
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o[0] / l, o[1] / l), hi = __floats2bfloat162_rn(o[2] / l, o[3] / l);
    *out = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
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

size_t attn_tree_bytes(const KvBatch &, int, int, int) { return 256; }

cudaError_t launch_attn_tree(const AttnTreeArgs &a, cudaStream_t s, const char **) {
    const dim3 grid((a.n * a.own.n_kv * a.group + kAttnWarps - 1) / kAttnWarps, a.own.n_seq), block(32 * kAttnWarps);
    return a.own.format == kKvE4m3 ? launch_pdl(attn_tree_kernel<true>, grid, block, 0, s, a)
                                   : launch_pdl(attn_tree_kernel<false>, grid, block, 0, s, a);
}

}  // namespace tfk
