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
// rows of 40 heads take 62 us (5.4 TB/s; a copy reaches 6.8).  A lane for 4
// elements, partners by shuffle and one element an instruction took 95 us, 68
// without the next heads' loads under way.
__device__ __forceinline__ void sincos_turns(unsigned long long frac, float &c, float &s) {
    const float half_turns = __int2float_rn(int(frac >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
}

constexpr int kRopeSteps = 2;   // pairs of heads a warp turns while as many are on their way

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
__global__ void __launch_bounds__(256, FP32 ? 2 : 3) qk_norm_rope_kernel(QkNormRopeArgs a, int heads_per_warp, int runs) {
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
    uint4 ahead[kRopeSteps][FP32 ? 2 : 1];      // the next heads, on their way while these are turned
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < kRopeSteps; ++u) {
            const int hu = h + 2 * u;
            if (hu >= h1) continue;
            if constexpr (FP32) {
                const float *from = reinterpret_cast<const float *>(src) + hu * kHeadDim;
                ahead[u][0] = __ldg(reinterpret_cast<const uint4 *>(from + e0));
                ahead[u][1] = __ldg(reinterpret_cast<const uint4 *>(from + e1));
            } else {    // not the read-only path: the caller may rotate rows in place
                const uint16_t *from = reinterpret_cast<const uint16_t *>(src) + hu * kHeadDim;
                const uint2 lo = *reinterpret_cast<const uint2 *>(from + e0), hi = *reinterpret_cast<const uint2 *>(from + e1);
                ahead[u][0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
    };
    load(h0 + half);
    for (int h = h0 + half; h < h1 + half; h += 2 * kRopeSteps) {
        uint4 x[kRopeSteps][FP32 ? 2 : 1];
#pragma unroll
        for (int u = 0; u < kRopeSteps; ++u) {
            x[u][0] = ahead[u][0];
            if constexpr (FP32) x[u][1] = ahead[u][1];
        }
        load(h + 2 * kRopeSteps);
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
// A CTA takes some rows of one sequence, all heads; 16 lanes move a row's K and V
// vectors of one head, 16 bytes of bf16 a lane each, two heads in flight.
// Consecutive half warps take consecutive heads of a row (which the rows hold
// together); a head's entries of consecutive rows are one CTA's.  HBM bounds both
// where there are many rows: 32767 rows of 8 heads, E4M3, are written and read back
// in 69 us (5.8 TB/s; 117 us with an integer division per vector's place).
constexpr int kVecUnroll = 2, kVecThreads = 256, kVecHalfWarps = kVecThreads / 16;

int rows_per_cta(int n_kv) { return n_kv < 64 ? 64 / n_kv : 1; }

// The (row, head) places of one half warp, in steps of kVecHalfWarps.
struct Places {
    int r, j, dr, dj, n_kv;
    __device__ __forceinline__ explicit Places(int n_kv_) : n_kv(n_kv_) {
        const int at = threadIdx.x >> 4;
        r = at / n_kv;
        j = at - r * n_kv;
        dr = kVecHalfWarps / n_kv;
        dj = kVecHalfWarps - dr * n_kv;
    }
    __device__ __forceinline__ void step() {
        r += dr;
        j += dj;
        if (j >= n_kv) {
            j -= n_kv;
            ++r;
        }
    }
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// One vector's 16-byte share of a lane -> its eight codes; s: the vector's scale byte.
__device__ __forceinline__ uint2 e4m3_codes(const uint4 &x, int &s) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = max_u16x2(max_u16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), max_u16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    const uint32_t peers = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(peers, m, o));
    s = e4m3_scale_byte(max(m & 0xFFFFu, m >> 16));
    if (s == kScaleNan) return make_uint2(0u, 0u);
    const float inv = __uint_as_float(uint32_t(254 - s) << 23);    // 2^-e
    uint32_t code[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        // bytes 0, 2 | 1, 3 of a word hold elements 0, 1 | 2, 3
        const uint32_t a = w[2 * e], d = w[2 * e + 1];
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(a << 16) * inv, __uint_as_float(d << 16) * inv),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(__uint_as_float(a & 0xFFFF0000u) * inv, __uint_as_float(d & 0xFFFF0000u) * inv), __NV_SATFINITE, __NV_E4M3);
        code[e] = lo | (hi << 16);
    }
    return make_uint2(code[0], code[1]);
}

template <bool E4M3>
__global__ void __launch_bounds__(kVecThreads) kv_store_kernel(KvBatch c, const uint16_t *k_new, const uint16_t *v_new,
                                                               int ld, int R, int rows_cta, const int64_t *pos, int *err) {
    grid_dependency_wait();     // the rows come from the preceding grid
    grid_launch_dependents();
    const int lane = threadIdx.x & 15, b = blockIdx.y, r0 = blockIdx.x * rows_cta, rows = min(rows_cta, R - r0);
    const long long p = seq_position(pos, b, R, c.max_len, err, blockIdx.x == 0 && threadIdx.x == 0);
    if (p < 0) return;
    const size_t row0 = ((size_t)b * R + r0) * ld + 8 * lane;
    const long long t0 = p + r0;
    Places at(c.n_kv);
    while (at.r < rows) {
        uint4 x[kVecUnroll][2];
        size_t entry[kVecUnroll];
        bool any[kVecUnroll];
#pragma unroll
        for (int i = 0; i < kVecUnroll; ++i) {
            any[i] = at.r < rows;
            if (any[i]) {
                const size_t from = row0 + (size_t)at.r * ld + at.j * kHeadDim;
                x[i][0] = *reinterpret_cast<const uint4 *>(k_new + from);
                x[i][1] = *reinterpret_cast<const uint4 *>(v_new + from);
                entry[i] = (size_t)(b * c.n_kv + at.j) * c.max_len + (size_t)(t0 + at.r);
            }
            at.step();
        }
#pragma unroll
        for (int i = 0; i < kVecUnroll; ++i) {
            if (!any[i]) break;
            if constexpr (!E4M3) {
                const size_t to = entry[i] * kHeadDim + ((lane ^ int(entry[i] & 7)) << 3);     // max_len % 8 = 0
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(c.k) + to) = x[i][0];
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(c.v) + to) = x[i][1];
            } else {
                const size_t to = entry[i] * kHeadDim + 16 * (lane & 7) + 8 * (lane >> 3);
                int sk, sv;
                const uint2 ck = e4m3_codes(x[i][0], sk), cv = e4m3_codes(x[i][1], sv);
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(c.k) + to) = ck;
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(c.v) + to) = cv;
                if (lane == 0) c.k_scale[entry[i]] = uint8_t(sk);
                if (lane == 1) c.v_scale[entry[i]] = uint8_t(sv);
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
    const size_t row0 = ((size_t)b * R + r0) * ld + 8 * lane;
    const long long t0 = p + r0;
    Places at(c.n_kv);
    while (at.r < rows) {
        uint4 x[kVecUnroll][2];
        uint32_t f[kVecUnroll][2];
        size_t to[kVecUnroll];
        bool any[kVecUnroll];
#pragma unroll
        for (int i = 0; i < kVecUnroll; ++i) {
            any[i] = at.r < rows;
            x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
            to[i] = row0 + (size_t)at.r * ld + at.j * kHeadDim;
            if (any[i] && p >= 0) {
                const size_t entry = (size_t)(b * c.n_kv + at.j) * c.max_len + (size_t)(t0 + at.r);
                if constexpr (!E4M3) {
                    const size_t from = entry * kHeadDim + ((lane ^ int(entry & 7)) << 3);      // max_len % 8 = 0
                    x[i][0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(c.k) + from);
                    x[i][1] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(c.v) + from);
                } else {
                    const size_t from = entry * kHeadDim + 16 * (lane & 7) + 8 * (lane >> 3);
                    const uint2 wk = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(c.k) + from);
                    const uint2 wv = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(c.v) + from);
                    x[i][0].x = wk.x, x[i][0].y = wk.y, x[i][1].x = wv.x, x[i][1].y = wv.y;
                    f[i][0] = c.k_scale[entry];
                    f[i][1] = c.v_scale[entry];
                }
            }
            at.step();
        }
#pragma unroll
        for (int i = 0; i < kVecUnroll; ++i) {
            if (!any[i]) break;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                uint4 y = x[i][w];
                if (E4M3 && p >= 0) {
                    const uint32_t factor = e4m3_factor(f[i][w]);
                    e4m3_expand(x[i][w].x, factor, y.x, y.y);
                    e4m3_expand(x[i][w].y, factor, y.z, y.w);
                }
                *reinterpret_cast<uint4 *>((w ? v_out : k_out) + to[i]) = y;
            }
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
