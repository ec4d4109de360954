// Per-head RMSNorm with position rotation, and the writes and reads of a batch
// of KV caches.  Every kernel here moves each byte once, so HBM bounds it where
// there are many rows and the launch where there are few.
#include "kv_batch.cuh"

#include "w4_gemm.cuh"

namespace tfk {

namespace {

// ------------------------------------------------------- norm and rotation
// One warp takes one row and a run of its heads, lane l elements 4l .. 4l + 3.
// cos and sin of the row's position are formed once per warp and reused for
// every head of the run.  The angle is counted in turns: position * turns[i]
// modulo 2^64 is the exact fraction of a turn of a 64-bit fixed-point
// frequency, whatever the position, and its top 32 bits go to sincospi as an
// fp32 in [-1, 1) half turns (off by at most 2^-25 half turns).
__device__ __forceinline__ void sincos_turns(unsigned long long frac, float &c, float &s) {
    const float half_turns = __int2float_rn(int(frac >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
}

constexpr int kRopeHeads = 4;   // heads a warp has in flight at a time

template <bool FP32>
__device__ __forceinline__ float4 load4(const void *x, size_t at) {
    if constexpr (FP32) {
        return __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(x) + at));
    } else {
        // not the read-only path: the caller may rotate rows in place
        const uint2 b = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(x) + at);
        return make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u),
                           __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xFFFF0000u));
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float4 weights4(const uint16_t *w, int lane) {
    const uint2 b = __ldg(reinterpret_cast<const uint2 *>(w) + lane);
    return make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u), __uint_as_float(b.y << 16),
                       __uint_as_float(b.y & 0xFFFF0000u));
}

template <bool FP32>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(QkNormRopeArgs a, int heads_per_warp, int runs) {
    grid_dependency_wait();     // x comes from the preceding grid
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const long long row = item / runs;
    if (row >= (long long)a.n_seq * a.R) return;
    const int H = a.n_q + a.n_k + a.n_v, n_rot = a.n_q + a.n_k;
    const int h0 = int(item % runs) * heads_per_warp, h1 = min(H, h0 + heads_per_warp);

    // lane's angles: element 4l + i turns by turns[...] (halves: pair (d, d + rot/2)
    // shares frequency d; adjacent: pair (2d, 2d + 1) shares frequency d)
    const bool rotated = 4 * lane < a.rot;
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    int partner = lane;
    if (rotated && h0 < n_rot) {
        const int b = int(row / a.R), r = int(row % a.R);
        const unsigned long long p = (unsigned long long)(a.pos[b] + a.pos_offset + r);
        if (a.adjacent) {
            const ulonglong2 t = __ldg(reinterpret_cast<const ulonglong2 *>(a.turns) + lane);
            sincos_turns(p * t.x, c[0], s[1]);
            sincos_turns(p * t.y, c[2], s[3]);
            c[1] = c[0];
            c[3] = c[2];
            s[0] = -s[1];
            s[2] = -s[3];
        } else {
            const int lanes = a.rot / 8;    // lanes of the first half
            const bool upper = lane >= lanes;
            const int l = upper ? lane - lanes : lane;
            partner = upper ? l : lane + lanes;
            const ulonglong2 t0 = __ldg(reinterpret_cast<const ulonglong2 *>(a.turns) + 2 * l);
            const ulonglong2 t1 = __ldg(reinterpret_cast<const ulonglong2 *>(a.turns) + 2 * l + 1);
            sincos_turns(p * t0.x, c[0], s[0]);
            sincos_turns(p * t0.y, c[1], s[1]);
            sincos_turns(p * t1.x, c[2], s[2]);
            sincos_turns(p * t1.y, c[3], s[3]);
            if (!upper) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = -s[i];
            }
        }
    }
    float4 wq = make_float4(1.f, 1.f, 1.f, 1.f), wk = wq;
    if (a.wq) {
        wq = weights4(a.wq, lane);
        wk = weights4(a.wk, lane);
    }
    for (int h = h0; h < h1; h += kRopeHeads) {
        float4 v[kRopeHeads];
#pragma unroll
        for (int u = 0; u < kRopeHeads; ++u)
            if (h + u < h1) v[u] = load4<FP32>(a.x, (size_t)row * a.ldx + (size_t)(h + u) * kHeadDim + 4 * lane);
#pragma unroll
        for (int u = 0; u < kRopeHeads; ++u) {
            if (h + u >= h1) break;
            float4 t = v[u];
            if (h + u < n_rot) {
                if (a.wq) {
                    float ss = fmaf(t.x, t.x, fmaf(t.y, t.y, fmaf(t.z, t.z, t.w * t.w)));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                    const float inv = 1.0f / sqrtf(fmaf(ss, 1.0f / kHeadDim, a.eps));
                    const float4 w = h + u < a.n_q ? wq : wk;
                    t.x = t.x * inv * w.x;
                    t.y = t.y * inv * w.y;
                    t.z = t.z * inv * w.z;
                    t.w = t.w * inv * w.w;
                }
                if (a.rot > 0) {
                    float4 o;
                    if (a.adjacent) {
                        o = make_float4(t.y, t.x, t.w, t.z);
                    } else {
                        o.x = __shfl_sync(0xFFFFFFFFu, t.x, partner);
                        o.y = __shfl_sync(0xFFFFFFFFu, t.y, partner);
                        o.z = __shfl_sync(0xFFFFFFFFu, t.z, partner);
                        o.w = __shfl_sync(0xFFFFFFFFu, t.w, partner);
                    }
                    if (rotated) {
                        t.x = fmaf(t.x, c[0], o.x * s[0]);
                        t.y = fmaf(t.y, c[1], o.y * s[1]);
                        t.z = fmaf(t.z, c[2], o.z * s[2]);
                        t.w = fmaf(t.w, c[3], o.w * s[3]);
                    }
                }
            }
            *reinterpret_cast<uint2 *>(a.y + (size_t)row * a.ldy + (size_t)(h + u) * kHeadDim + 4 * lane) =
                make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
        }
    }
}

// ------------------------------------------------------- cache writes and reads
// 16 lanes move one vector (K or V of one row and head), 16 bytes of bf16 each.
// Vectors are taken head-major within a sequence, rows ascending, so that
// neighbouring half warps touch neighbouring cache entries.
struct Vec {
    int b, j, which;
    long long row, r;
};

__device__ __forceinline__ bool vec_of(long long i, const KvBatch &c, int R, Vec &v) {
    const long long per_seq = 2LL * R * c.n_kv;
    if (i >= per_seq * c.n_seq) return false;
    v.b = int(i / per_seq);
    i -= v.b * per_seq;
    v.which = int(i & 1);
    i >>= 1;
    v.j = int(i % c.n_kv);
    v.r = i / c.n_kv;
    v.row = (long long)v.b * R + v.r;
    return true;
}

template <bool E4M3>
__global__ void __launch_bounds__(256) kv_store_kernel(KvBatch c, const uint16_t *k_new, const uint16_t *v_new, int ld,
                                                       int R, const int64_t *pos, int *err) {
    grid_dependency_wait();     // the rows come from the preceding grid
    grid_launch_dependents();
    Vec u;
    const int lane = threadIdx.x & 15;
    if (!vec_of((long long)blockIdx.x * 16 + (threadIdx.x >> 4), c, R, u)) return;
    const long long p = seq_position(pos, u.b, R, c.max_len, err, u.r == 0 && lane == 0);
    if (p < 0) return;
    const long long t = p + u.r;
    const uint4 x = *reinterpret_cast<const uint4 *>((u.which ? v_new : k_new) + (size_t)u.row * ld + u.j * kHeadDim +
                                                     8 * lane);
    const size_t entry = ((size_t)u.b * c.n_kv + u.j) * c.max_len + (size_t)t;
    if constexpr (!E4M3) {
        uint16_t *dst = static_cast<uint16_t *>(u.which ? c.v : c.k) + entry * kHeadDim + ((lane ^ int(t & 7)) << 3);
        *reinterpret_cast<uint4 *>(dst) = x;
    } else {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
        const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(half, m, o));
        const int s = e4m3_scale_byte(m);
        uint32_t code[2] = {0u, 0u};
        if (s != kScaleNan) {
            const float inv = __uint_as_float(uint32_t(254 - s) << 23);    // 2^-e
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // bytes 0, 2 | 1, 3 of a word hold elements 0, 1 | 2, 3
                const uint32_t a = w[2 * i], b = w[2 * i + 1];
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(a << 16) * inv,
                                                                         __uint_as_float(b << 16) * inv),
                                                             __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(a & 0xFFFF0000u) * inv,
                                                                         __uint_as_float(b & 0xFFFF0000u) * inv),
                                                             __NV_SATFINITE, __NV_E4M3);
                code[i] = lo | (hi << 16);
            }
        }
        uint8_t *dst = static_cast<uint8_t *>(u.which ? c.v : c.k) + entry * kHeadDim + 16 * (lane & 7) + 8 * (lane >> 3);
        *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
        if (lane == 0) (u.which ? c.v_scale : c.k_scale)[entry] = uint8_t(s);
    }
}

template <bool E4M3>
__global__ void __launch_bounds__(256) kv_load_kernel(KvBatch c, const int64_t *pos, int R, uint16_t *k_out,
                                                      uint16_t *v_out, int ld, int *err) {
    grid_dependency_wait();     // the entries come from the preceding grid
    grid_launch_dependents();
    Vec u;
    const int lane = threadIdx.x & 15;
    if (!vec_of((long long)blockIdx.x * 16 + (threadIdx.x >> 4), c, R, u)) return;
    const long long p = seq_position(pos, u.b, R, c.max_len, err, u.r == 0 && lane == 0);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (p >= 0) {
        const long long t = p + u.r;
        const size_t entry = ((size_t)u.b * c.n_kv + u.j) * c.max_len + (size_t)t;
        if constexpr (!E4M3) {
            const uint16_t *src = static_cast<const uint16_t *>(u.which ? c.v : c.k) + entry * kHeadDim +
                                  ((lane ^ int(t & 7)) << 3);
            x = *reinterpret_cast<const uint4 *>(src);
        } else {
            const uint8_t *src = static_cast<const uint8_t *>(u.which ? c.v : c.k) + entry * kHeadDim +
                                 16 * (lane & 7) + 8 * (lane >> 3);
            const uint2 w = *reinterpret_cast<const uint2 *>(src);
            const uint32_t f = e4m3_factor((u.which ? c.v_scale : c.k_scale)[entry]);
            e4m3_expand(w.x, f, x.x, x.y);
            e4m3_expand(w.y, f, x.z, x.w);
        }
    }
    *reinterpret_cast<uint4 *>((u.which ? v_out : k_out) + (size_t)u.row * ld + u.j * kHeadDim + 8 * lane) = x;
}

unsigned vec_blocks(const KvBatch &c, int R) {
    return unsigned((2LL * c.n_seq * R * c.n_kv + 15) / 16);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs &a, cudaStream_t s) {
    const int H = a.n_q + a.n_k + a.n_v;
    const long long rows = (long long)a.n_seq * a.R;
    int hpw = 1;
    while (hpw < 16 && rows * ((H + hpw - 1) / hpw) > 32LL * device_sm_count()) hpw *= 2;
    const int runs = (H + hpw - 1) / hpw;
    const unsigned blocks = unsigned((rows * runs + 7) / 8);
    return a.x_fp32 ? launch_pdl(qk_norm_rope_kernel<true>, dim3(blocks), dim3(256), 0, s, a, hpw, runs)
                    : launch_pdl(qk_norm_rope_kernel<false>, dim3(blocks), dim3(256), 0, s, a, hpw, runs);
}

cudaError_t launch_kv_store(const KvBatch &c, const uint16_t *k_new, const uint16_t *v_new, int ld, int R,
                            const int64_t *pos, int *err, cudaStream_t s) {
    const dim3 grid(vec_blocks(c, R));
    return c.format == kKvE4m3
               ? launch_pdl(kv_store_kernel<true>, grid, dim3(256), 0, s, c, k_new, v_new, ld, R, pos, err)
               : launch_pdl(kv_store_kernel<false>, grid, dim3(256), 0, s, c, k_new, v_new, ld, R, pos, err);
}

cudaError_t launch_kv_load(const KvBatch &c, const int64_t *pos, int R, uint16_t *k_out, uint16_t *v_out, int ld,
                           int *err, cudaStream_t s) {
    const dim3 grid(vec_blocks(c, R));
    return c.format == kKvE4m3 ? launch_pdl(kv_load_kernel<true>, grid, dim3(256), 0, s, c, pos, R, k_out, v_out, ld, err)
                               : launch_pdl(kv_load_kernel<false>, grid, dim3(256), 0, s, c, pos, R, k_out, v_out, ld,
                                            err);
}

}  // namespace tfk
