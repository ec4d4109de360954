// Per-head RMSNorm with position rotation, and the writes and reads of a batch
// of KV caches.  Every kernel here moves each byte once, so HBM bounds it where
// there are many rows and the launch where there are few.
#include "kv_batch.cuh"

#include "w4_gemm.cuh"

namespace tfk {

namespace {

// ------------------------------------------------------- norm and rotation
// One warp takes one row and a run of its heads, two at a time: 16 lanes a head,
// 8 elements a lane, as two chunks of 4 chosen so that both elements of every
// rotated pair are one lane's (pairs of halves: chunk i and chunk i + rot/8;
// adjacent pairs, and elements past rot: neighbouring chunks).  The lane's four
// cosines and sines are formed once per warp and reused for every head.  The
// angle is counted in turns: position * turns[i] modulo 2^64 is the exact
// fraction of a turn of a 64-bit fixed-point frequency, whatever the position, and
// its top 32 bits go to sincospi as an fp32 in [-1, 1) half turns (off by at
// most 2^-25 half turns).  HBM bounds it where there are many rows: 16383 bf16
// rows of 40 heads in PROMPT_US us (PROMPT_GBS of 6.78 TB/s copy); four lanes' worth of
// shuffles fewer and two elements an instruction took it there from 95 us.
__device__ __forceinline__ void sincos_turns(unsigned long long frac, float &c, float &s) {
    const float half_turns = __int2float_rn(int(frac >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
}

constexpr int kRopeSteps = 4;   // pairs of heads a warp has in flight

__device__ __forceinline__ uint64_t widen2(uint32_t w) {       // two bf16 -> two fp32
    return uint64_t(w << 16) | (uint64_t(w & 0xFFFF0000u) << 32);
}
__device__ __forceinline__ uint32_t narrow2(uint64_t v) {
    float a, b;
    unpack2(v, a, b);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <bool FP32>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(QkNormRopeArgs a, int heads_per_warp, int runs) {
    grid_dependency_wait();     // x comes from the preceding grid
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, half = lane >> 4, sub = lane & 15;
    const unsigned item = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const unsigned row = item / unsigned(runs);
    if (row >= unsigned(a.n_seq) * unsigned(a.R)) return;
    const int H = a.n_q + a.n_k + a.n_v, n_rot = a.n_q + a.n_k;
    const int h0 = int(item - row * runs) * heads_per_warp, h1 = min(H, h0 + heads_per_warp);

    const int pairs = a.rot / 8;                        // lanes whose elements turn
    const bool turning = sub < pairs;
    const bool halves = turning && !a.adjacent;
    const int e0 = 4 * (halves ? sub : 2 * sub), e1 = halves ? e0 + a.rot / 2 : e0 + 4;   // first elements of the chunks
    // out_k = v_k * C_k + u_k * S_k on pairs of elements, u = the other chunk's (halves)
    // or the swapped pair (adjacent)
    uint64_t C[4], S[4];
    if (turning && h0 < n_rot) {
        const unsigned b = row / unsigned(a.R), r = row - b * a.R;
        const unsigned long long p = (unsigned long long)(a.pos[b] + a.pos_offset + r);
        const ulonglong2 t0 = __ldg(reinterpret_cast<const ulonglong2 *>(a.turns) + 2 * sub);
        const ulonglong2 t1 = __ldg(reinterpret_cast<const ulonglong2 *>(a.turns) + 2 * sub + 1);
        float c[4], s[4];
        sincos_turns(p * t0.x, c[0], s[0]);
        sincos_turns(p * t0.y, c[1], s[1]);
        sincos_turns(p * t1.x, c[2], s[2]);
        sincos_turns(p * t1.y, c[3], s[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 2 * (i & 1);
            C[i] = halves ? pack2(c[j], c[j + 1]) : pack2(c[i], c[i]);
            S[i] = halves ? (i < 2 ? pack2(-s[j], -s[j + 1]) : pack2(s[j], s[j + 1])) : pack2(-s[i], s[i]);
        }
    }
    uint64_t wq[4], wk[4];
    if (a.wq) {
        const uint2 q0 = __ldg(reinterpret_cast<const uint2 *>(a.wq + e0)), q1 = __ldg(reinterpret_cast<const uint2 *>(a.wq + e1));
        const uint2 k0 = __ldg(reinterpret_cast<const uint2 *>(a.wk + e0)), k1 = __ldg(reinterpret_cast<const uint2 *>(a.wk + e1));
        wq[0] = widen2(q0.x), wq[1] = widen2(q0.y), wq[2] = widen2(q1.x), wq[3] = widen2(q1.y);
        wk[0] = widen2(k0.x), wk[1] = widen2(k0.y), wk[2] = widen2(k1.x), wk[3] = widen2(k1.y);
    }
    const char *src = static_cast<const char *>(a.x) + (size_t)row * a.ldx * (FP32 ? 4 : 2);
    uint16_t *dst = a.y + (size_t)row * a.ldy;
    for (int h = h0 + half; h < h1 + half; h += 2 * kRopeSteps) {
        uint4 x[kRopeSteps][FP32 ? 2 : 1];
#pragma unroll
        for (int u = 0; u < kRopeSteps; ++u) {
            const int hu = h + 2 * u;
            if (hu >= h1) continue;
            if constexpr (FP32) {
                const float *from = reinterpret_cast<const float *>(src) + hu * kHeadDim;
                x[u][0] = __ldg(reinterpret_cast<const uint4 *>(from + e0));
                x[u][1] = __ldg(reinterpret_cast<const uint4 *>(from + e1));
            } else {    // not the read-only path: the caller may rotate rows in place
                const uint16_t *from = reinterpret_cast<const uint16_t *>(src) + hu * kHeadDim;
                const uint2 lo = *reinterpret_cast<const uint2 *>(from + e0), hi = *reinterpret_cast<const uint2 *>(from + e1);
                x[u][0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
#pragma unroll
        for (int u = 0; u < kRopeSteps; ++u) {
            const int hu = h + 2 * u;
            if (hu - half >= h1) break;         // neither half warp has a head left
            uint64_t v[4];
            if constexpr (FP32) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    v[2 * i] = uint64_t(x[u][i].x) | (uint64_t(x[u][i].y) << 32);
                    v[2 * i + 1] = uint64_t(x[u][i].z) | (uint64_t(x[u][i].w) << 32);
                }
            } else {
                v[0] = widen2(x[u][0].x), v[1] = widen2(x[u][0].y), v[2] = widen2(x[u][0].z), v[3] = widen2(x[u][0].w);
            }
            const bool normed = a.wq && hu < n_rot;
            if (__any_sync(0xFFFFFFFFu, normed)) {
                float s0, s1;
                unpack2(fma2(v[0], v[0], fma2(v[1], v[1], fma2(v[2], v[2], mul2(v[3], v[3])))), s0, s1);
                float ss = s0 + s1;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                if (normed) {
                    const float inv = rsqrtf(fmaf(ss, 1.0f / kHeadDim, a.eps));
                    const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = mul2(mul2(v[i], inv2), hu < a.n_q ? wq[i] : wk[i]);
                }
            }
            if (turning && hu < n_rot) {
                uint64_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t other = halves ? v[i ^ 2] : (v[i] >> 32) | (v[i] << 32);
                    o[i] = fma2(v[i], C[i], mul2(other, S[i]));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = o[i];
            }
            if (hu < h1) {
                *reinterpret_cast<uint2 *>(dst + hu * kHeadDim + e0) = make_uint2(narrow2(v[0]), narrow2(v[1]));
                *reinterpret_cast<uint2 *>(dst + hu * kHeadDim + e1) = make_uint2(narrow2(v[2]), narrow2(v[3]));
            }
        }
    }
}

// ------------------------------------------------------- cache writes and reads
// A CTA takes some rows of one sequence, all heads, K and V; 16 lanes move one
// vector (K or V of one row and head), 16 bytes of bf16 each, four vectors in
// flight.  Consecutive half warps take consecutive heads of a row (the rows are
// contiguous); a head's entries of consecutive rows are written by one CTA.
constexpr int kVecUnroll = 4, kVecThreads = 256, kVecHalfWarps = kVecThreads / 16;

int rows_per_cta(int n_kv) { return n_kv < 32 ? 32 / n_kv : 1; }

struct Vec {
    int j, which, r;        // head, K or V, row within the CTA's
    bool any;
};
__device__ __forceinline__ Vec vec_of(int u, int n_kv, int rows) {
    Vec v;
    v.any = u < 2 * rows * n_kv;
    v.which = u >= rows * n_kv;
    if (v.which) u -= rows * n_kv;
    v.r = idx_div(u, n_kv);
    v.j = u - v.r * n_kv;
    return v;
}

template <bool E4M3>
__global__ void __launch_bounds__(kVecThreads) kv_store_kernel(KvBatch c, const uint16_t *k_new, const uint16_t *v_new,
                                                               int ld, int R, int rows_cta, const int64_t *pos, int *err) {
    grid_dependency_wait();     // the rows come from the preceding grid
    grid_launch_dependents();
    const int lane = threadIdx.x & 15, b = blockIdx.y, r0 = blockIdx.x * rows_cta, rows = min(rows_cta, R - r0);
    const long long p = seq_position(pos, b, R, c.max_len, err, blockIdx.x == 0 && threadIdx.x == 0);
    if (p < 0) return;
    const size_t row0 = (size_t)b * R + r0;
    for (int u0 = threadIdx.x >> 4; u0 < 2 * rows * c.n_kv; u0 += kVecUnroll * kVecHalfWarps) {
        uint4 x[kVecUnroll];
#pragma unroll
        for (int i = 0; i < kVecUnroll; ++i) {
            const Vec u = vec_of(u0 + i * kVecHalfWarps, c.n_kv, rows);
            if (u.any)
                x[i] = *reinterpret_cast<const uint4 *>((u.which ? v_new : k_new) + (row0 + u.r) * ld + u.j * kHeadDim + 8 * lane);
        }
#pragma unroll
        for (int i = 0; i < kVecUnroll; ++i) {
            const Vec u = vec_of(u0 + i * kVecHalfWarps, c.n_kv, rows);
            if (!u.any) break;
            const long long t = p + r0 + u.r;
            const size_t entry = ((size_t)b * c.n_kv + u.j) * c.max_len + (size_t)t;
            if constexpr (!E4M3) {
                uint16_t *dst = static_cast<uint16_t *>(u.which ? c.v : c.k) + entry * kHeadDim + ((lane ^ int(t & 7)) << 3);
                *reinterpret_cast<uint4 *>(dst) = x[i];
            } else {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
                const uint32_t peers = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(peers, m, o));
                const int s = e4m3_scale_byte(m);
                uint32_t code[2] = {0u, 0u};
                if (s != kScaleNan) {
                    const float inv = __uint_as_float(uint32_t(254 - s) << 23);    // 2^-e
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // bytes 0, 2 | 1, 3 of a word hold elements 0, 1 | 2, 3
                        const uint32_t a = w[2 * e], d = w[2 * e + 1];
                        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                            make_float2(__uint_as_float(a << 16) * inv, __uint_as_float(d << 16) * inv), __NV_SATFINITE, __NV_E4M3);
                        const uint32_t hi =
                            __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(a & 0xFFFF0000u) * inv,
                                                                 __uint_as_float(d & 0xFFFF0000u) * inv),
                                                     __NV_SATFINITE, __NV_E4M3);
                        code[e] = lo | (hi << 16);
                    }
                }
                uint8_t *dst = static_cast<uint8_t *>(u.which ? c.v : c.k) + entry * kHeadDim + 16 * (lane & 7) + 8 * (lane >> 3);
                *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
                if (lane == 0) (u.which ? c.v_scale : c.k_scale)[entry] = uint8_t(s);
            }
        }
    }
}

template <bool E4M3>
__global__ void __launch_bounds__(kVecThreads) kv_load_kernel(KvBatch c, const int64_t *pos, int R, int rows_cta,
                                                              uint16_t *k_out, uint16_t *v_out, int ld, int *err) {
    grid_dependency_wait();     // the entries come from the preceding grid
    grid_launch_dependents();
    const int lane = threadIdx.x & 15, b = blockIdx.y, r0 = blockIdx.x * rows_cta, rows = min(rows_cta, R - r0);
    const long long p = seq_position(pos, b, R, c.max_len, err, blockIdx.x == 0 && threadIdx.x == 0);
    const size_t row0 = (size_t)b * R + r0;
    for (int u0 = threadIdx.x >> 4; u0 < 2 * rows * c.n_kv; u0 += kVecUnroll * kVecHalfWarps) {
        uint4 x[kVecUnroll];
        uint32_t f[kVecUnroll];
#pragma unroll
        for (int i = 0; i < kVecUnroll; ++i) {
            const Vec u = vec_of(u0 + i * kVecHalfWarps, c.n_kv, rows);
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            f[i] = 0u;
            if (!u.any || p < 0) continue;
            const long long t = p + r0 + u.r;
            const size_t entry = ((size_t)b * c.n_kv + u.j) * c.max_len + (size_t)t;
            if constexpr (!E4M3) {
                x[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(u.which ? c.v : c.k) + entry * kHeadDim +
                                                        ((lane ^ int(t & 7)) << 3));
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(u.which ? c.v : c.k) +
                                                                 entry * kHeadDim + 16 * (lane & 7) + 8 * (lane >> 3));
                x[i].x = w.x;
                x[i].y = w.y;
                f[i] = (u.which ? c.v_scale : c.k_scale)[entry];
            }
        }
#pragma unroll
        for (int i = 0; i < kVecUnroll; ++i) {
            const Vec u = vec_of(u0 + i * kVecHalfWarps, c.n_kv, rows);
            if (!u.any) break;
            uint4 y = x[i];
            if (E4M3 && p >= 0) {
                const uint32_t factor = e4m3_factor(f[i]);
                e4m3_expand(x[i].x, factor, y.x, y.y);
                e4m3_expand(x[i].y, factor, y.z, y.w);
            }
            *reinterpret_cast<uint4 *>((u.which ? v_out : k_out) + (row0 + u.r) * ld + u.j * kHeadDim + 8 * lane) = y;
        }
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs &a, cudaStream_t s) {
    // heads a warp takes: as many as leave 32 warps an SM, so that few rows are
    // spread over the GPU and many rows form their cosines once
    const int H = a.n_q + a.n_k + a.n_v;
    const long long rows = (long long)a.n_seq * a.R, enough = 32LL * device_sm_count();
    int hpw = 2;
    while (hpw < H && rows * ((H + 2 * hpw - 1) / (2 * hpw)) >= enough) hpw *= 2;
    const int runs = (H + hpw - 1) / hpw;
    const unsigned blocks = unsigned((rows * runs + 7) / 8);
    return a.x_fp32 ? launch_pdl(qk_norm_rope_kernel<true>, dim3(blocks), dim3(256), 0, s, a, hpw, runs)
                    : launch_pdl(qk_norm_rope_kernel<false>, dim3(blocks), dim3(256), 0, s, a, hpw, runs);
}

cudaError_t launch_kv_store(const KvBatch &c, const uint16_t *k_new, const uint16_t *v_new, int ld, int R,
                            const int64_t *pos, int *err, cudaStream_t s) {
    const int rows = rows_per_cta(c.n_kv);
    const dim3 grid((R + rows - 1) / rows, c.n_seq), block(kVecThreads);
    return c.format == kKvE4m3
               ? launch_pdl(kv_store_kernel<true>, grid, block, 0, s, c, k_new, v_new, ld, R, rows, pos, err)
               : launch_pdl(kv_store_kernel<false>, grid, block, 0, s, c, k_new, v_new, ld, R, rows, pos, err);
}

cudaError_t launch_kv_load(const KvBatch &c, const int64_t *pos, int R, uint16_t *k_out, uint16_t *v_out, int ld,
                           int *err, cudaStream_t s) {
    const int rows = rows_per_cta(c.n_kv);
    const dim3 grid((R + rows - 1) / rows, c.n_seq), block(kVecThreads);
    return c.format == kKvE4m3
               ? launch_pdl(kv_load_kernel<true>, grid, block, 0, s, c, pos, R, rows, k_out, v_out, ld, err)
               : launch_pdl(kv_load_kernel<false>, grid, block, 0, s, c, pos, R, rows, k_out, v_out, ld, err);
}

}  // namespace tfk
