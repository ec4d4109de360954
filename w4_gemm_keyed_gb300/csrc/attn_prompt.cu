// Causal attention of whole prompts, packed one after the other.
//
// Row i of a sequence attends over its rows 0 .. i:
//   s_t = q . k_t / sqrt(128),  o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m).
#include <cuda_bf16.h>

#include "attn_prompt.cuh"

namespace tfk {

namespace {

constexpr float kScale = 0.08838834764831845f;      // 1 / sqrt(128)
constexpr int kWarps = 4;

__device__ __forceinline__ void eight(const uint16_t *p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// A warp per (row, query head): keys 32 at a time, a key per lane for the scores, four
// output columns per lane for the sums, all in fp32.
__global__ void __launch_bounds__(32 * kWarps) attn_prompt_kernel(AttnPromptArgs a) {
    __shared__ float s_q[kWarps][kHeadDim];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_q = a.n_kv * a.group;
    bool bad = false;
    for (int s = lane; s <= a.n_seq; s += 32) {
        const long long x = a.starts[s];
        bad |= x < 0 || x > a.rows || (s > 0 && x < a.starts[s - 1]);
    }
    if (__any_sync(0xFFFFFFFFu, bad)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(a.err, kDevBadPosition);
        return;
    }
    const long long unit = (long long)blockIdx.x * kWarps + warp;
    if (unit >= (long long)a.rows * n_q) return;
    const int row = int(unit / n_q), h = int(unit - (long long)row * n_q), j = h / a.group;
    if (row < a.starts[0] || row >= a.starts[a.n_seq]) return;
    int lo = 0, hi = a.n_seq - 1;       // last sequence that starts at or before the row
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.starts[mid] <= row)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int first = int(a.starts[lo]);
    const uint16_t *q = a.q + (size_t)row * a.ldq + h * kHeadDim;
    for (int i = lane; i < kHeadDim; i += 32) s_q[warp][i] = __uint_as_float(uint32_t(q[i]) << 16) * kScale;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t0 = first; t0 <= row; t0 += 32) {
        const int t = t0 + lane;
        float s = -INFINITY;
        if (t <= row) {
            s = 0.f;
            for (int c = 0; c < 16; ++c) {
                float x[8];
                eight(a.k + (size_t)t * a.ldk + j * kHeadDim + 8 * c, x);
                for (int i = 0; i < 8; ++i) s = fmaf(x[i], s_q[warp][8 * c + i], s);
            }
        }
        float top = s;
        for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
        top = fmaxf(top, m);
        const float scale = top == -INFINITY ? 1.f : expf(m - top), w = t <= row ? expf(s - top) : 0.f;
        float sum = w;
        for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
        l = l * scale + sum;
        m = top;
        for (int i = 0; i < 4; ++i) o[i] *= scale;
        const int keys = min(32, row - t0 + 1);
        for (int u = 0; u < keys; ++u) {
            const float wu = __shfl_sync(0xFFFFFFFFu, w, u);
            const uint2 p = *reinterpret_cast<const uint2 *>(a.v + (size_t)(t0 + u) * a.ldv + j * kHeadDim + 4 * lane);
            o[0] = fmaf(wu, __uint_as_float(p.x << 16), o[0]);
            o[1] = fmaf(wu, __uint_as_float(p.x & 0xFFFF0000u), o[1]);
            o[2] = fmaf(wu, __uint_as_float(p.y << 16), o[2]);
            o[3] = fmaf(wu, __uint_as_float(p.y & 0xFFFF0000u), o[3]);
        }
    }
    const __nv_bfloat162 x = __floats2bfloat162_rn(o[0] / l, o[1] / l), y = __floats2bfloat162_rn(o[2] / l, o[3] / l);
    reinterpret_cast<uint2 *>(a.out + (size_t)row * a.ldo + h * kHeadDim)[lane] =
        make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}

}  // namespace

cudaError_t launch_attn_prompt(const AttnPromptArgs &a, cudaStream_t s, const char **) {
    const long long units = (long long)a.rows * a.n_kv * a.group;
    return launch_pdl(attn_prompt_kernel, dim3(unsigned((units + kWarps - 1) / kWarps)), dim3(32 * kWarps), 0, s, a);
}

}  // namespace tfk
