// Attention of a batch of sequences that continue one prompt.
//
// Row r of sequence b (position pos[b] + r of its own cache) attends over the
// shared prefix's entries 0 .. P - 1 and its own entries 0 .. pos[b] + r:
//   s_t = q . k_t / sqrt(128),  o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m).
// One warp takes one query vector and walks its keys in ascending order with a
// running maximum m, weight sum l and output o in fp32.
#include "attn_batch.cuh"

namespace tfk {

namespace {

constexpr float kLog2eOverSqrtD = 0.12751743074439720f;   // log2(e) / sqrt(128)

__device__ __forceinline__ float4 entry4(const KvBatch &c, int which, size_t entry, long long t, int lane) {
    uint32_t lo, hi;
    if (c.format == kKvE4m3) {
        const uint8_t *p = static_cast<const uint8_t *>(which ? c.v : c.k) + entry * kHeadDim + e4m3_byte(4 * lane);
        e4m3_expand(*reinterpret_cast<const uint32_t *>(p), e4m3_factor((which ? c.v_scale : c.k_scale)[entry]), lo, hi);
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(which ? c.v : c.k) + entry * kHeadDim +
                            (((lane >> 1) ^ int(t & 7)) << 3) + 4 * (lane & 1);
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        lo = w.x;
        hi = w.y;
    }
    return make_float4(__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u), __uint_as_float(hi << 16),
                       __uint_as_float(hi & 0xFFFF0000u));
}

__global__ void __launch_bounds__(128) attn_batch_kernel(AttnBatchArgs a) {
    grid_dependency_wait();     // queries and entries come from the preceding grids
    grid_launch_dependents();
    const int n_q = a.own.n_kv * a.group, lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (item >= (long long)a.own.n_seq * a.R * n_q) return;
    const int h = int(item % n_q), j = h / a.group;
    const long long row = item / n_q;
    const int b = int(row / a.R), r = int(row % a.R);
    const long long p = seq_position(a.pos, b, a.R, a.own.max_len, a.err, lane == 0);
    uint2 *out = reinterpret_cast<uint2 *>(a.out + (size_t)row * a.ldo + (size_t)h * kHeadDim) + lane;
    if (p < 0) {
        *out = make_uint2(0u, 0u);
        return;
    }
    const uint2 qw = *(reinterpret_cast<const uint2 *>(a.q + (size_t)row * a.ldq + (size_t)h * kHeadDim) + lane);
    const float4 q = make_float4(__uint_as_float(qw.x << 16), __uint_as_float(qw.x & 0xFFFF0000u),
                                 __uint_as_float(qw.y << 16), __uint_as_float(qw.y & 0xFFFF0000u));
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto walk = [&](const KvBatch &c, size_t base, long long n) {
        for (long long t = 0; t < n; ++t) {
            const float4 k = entry4(c, 0, base + t, t, lane);
            float s = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, q.w * k.w)));
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, i);
            s *= kLog2eOverSqrtD;
            const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
            const float scale = exp2f(m - ref), w = exp2f(s - ref);
            const float4 v = entry4(c, 1, base + t, t, lane);
            l = fmaf(l, scale, w);
            o.x = fmaf(o.x, scale, w * v.x);
            o.y = fmaf(o.y, scale, w * v.y);
            o.z = fmaf(o.z, scale, w * v.z);
            o.w = fmaf(o.w, scale, w * v.w);
            m = mn;
        }
    };
    walk(a.prefix, (size_t)j * a.prefix.max_len, a.prefix_len);
    walk(a.own, ((size_t)b * a.own.n_kv + j) * a.own.max_len, p + r + 1);
    const __nv_bfloat162 lo = __floats2bfloat162_rn(__fdiv_rn(o.x, l), __fdiv_rn(o.y, l));
    const __nv_bfloat162 hi = __floats2bfloat162_rn(__fdiv_rn(o.z, l), __fdiv_rn(o.w, l));
    *out = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

}  // namespace

size_t attn_batch_bytes(const KvBatch &, int, int, int) { return 256; }

cudaError_t launch_attn_batch(const AttnBatchArgs &a, cudaStream_t s) {
    const long long items = (long long)a.own.n_seq * a.R * a.own.n_kv * a.group;
    return launch_pdl(attn_batch_kernel, dim3(unsigned((items + 3) / 4)), dim3(128), 0, s, a);
}

}  // namespace tfk
