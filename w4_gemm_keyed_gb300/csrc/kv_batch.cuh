// Rows of a batch of sequences on their way into attention: per-head RMSNorm
// with position rotation, and a batch of KV caches held as bf16 or E4M3.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "attention.cuh"
#include "tf_ptx.cuh"

namespace tfk {

constexpr int kKvE4m3 = 1;  // the other format, 0, is bf16

// n_seq caches of n_kv heads and max_len entries.  bf16: tf_kv_cache's layout
// per sequence.  E4M3: 128 codes per entry, one scale byte per entry and head.
struct KvBatch {
    void *k, *v;
    uint8_t *k_scale, *v_scale;
    int n_seq, n_kv, max_len, format;
};

// A sequence's first position: -1 marks an idle sequence, anything else outside
// [0, max_len - R] a bad one (reported; treated as idle).
__device__ __forceinline__ long long seq_position(const int64_t *pos, int b, int R, int max_len, int *err,
                                                  bool report) {
    const long long p = pos[b];
    if (p == -1) return -1;
    if (p < 0 || p > (long long)max_len - R) {
        if (report) set_error(err, kDevBadPosition);
        return -1;
    }
    return p;
}

// ---- E4M3 vectors -----------------------------------------------------------
// A vector of 128 is 128 codes and a scale byte s: value = code * 2^(s - 127),
// s = 255: every element is NaN.  The exponent e = s - 127 is the smallest in
// [-120, 7] with max|x| <= 448 * 2^e, so a power of two: scaling is exact, and
// code * 2^e has 4 significant bits and fits bf16 exactly.  Element d of an
// entry is stored at byte e4m3_byte(d): 16 bytes hold eight consecutive
// elements of the lower half and the eight 64 above them (so eight lanes that
// expand one entry write each half's eight 16-byte chunks without bank
// conflicts), and the middle two bytes of a 4-byte word are exchanged (so that
// expanding even and odd bytes gives pairs of neighbours).
__host__ __device__ constexpr int e4m3_byte(int d) {
    const int i = d & 3;
    return 16 * ((d & 63) >> 3) + 8 * (d >> 6) + (d & 4) + (i == 1 ? 2 : (i == 2 ? 1 : i));
}

constexpr int kE4m3MinExp = -120, kE4m3MaxExp = 7;
constexpr int kScaleNan = 255;    // its codes are zeros

// Scale byte of a vector whose largest bf16 magnitude has the bits m (sign
// cleared).  448 = 1.75 * 2^8.
__device__ __forceinline__ int e4m3_scale_byte(uint32_t m) {
    if (m >= 0x7F80u) return kScaleNan;
    const int e = int(m >> 7) - 127 - 8 + ((m & 0x7Fu) > 0x60u ? 1 : 0);
    return min(max(e, kE4m3MinExp), kE4m3MaxExp) + 127;
}

// bf16x2 factor that turns expanded codes (code * 2^-120) into values: 2^(s - 7),
// or infinity for the NaN mark, whose codes are zeros (0 * inf = NaN).
__device__ __forceinline__ uint32_t e4m3_factor(uint32_t s) { return min(s + 120u, 255u) * 0x00800080u; }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four codes of one 4-byte word -> four bf16 values (lo: elements 0, 1; hi: 2, 3).
// A code's exponent and mantissa bits, moved to bits 10..4 of a bf16, read as
// code * 2^-120 (subnormal codes as subnormal bf16); one exact product with the
// factor restores the value.  Left shifts are products, which leave the logic
// unit (half the multiply unit's rate) to the masks.
__device__ __forceinline__ void e4m3_expand(uint32_t w, uint32_t factor, uint32_t &lo, uint32_t &hi) {
    constexpr uint32_t kMagnitude = 0x07F007F0u, kSign = 0x80008000u;
    lo = mul_bf16x2(lop3_and_or(w * 256u, kSign, (w * 16u) & kMagnitude), factor);
    hi = mul_bf16x2(lop3_and_or(w, kSign, (w >> 4) & kMagnitude), factor);
}

// Two fp32 operations in one instruction, each rounded as the single one is.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    return uint64_t(__float_as_uint(a)) | (uint64_t(__float_as_uint(b)) << 32);
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    a = __uint_as_float(uint32_t(v));
    b = __uint_as_float(uint32_t(v >> 32));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

struct QkNormRopeArgs {
    const void *x;          // fp32 or bf16 [n_seq * R][ldx]
    int x_fp32, ldx;
    int n_seq, R, n_q, n_k, n_v;
    const uint16_t *wq, *wk;    // bf16 [128] each, or both null: no norm
    float eps;
    const uint64_t *turns;  // [rot / 2]: turns per position in units of 2^-64
    int rot, adjacent;
    const int64_t *pos;
    long long pos_offset;
    uint16_t *y;            // bf16 [n_seq * R][ldy]
    int ldy;
};

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs &a, cudaStream_t s);
// entries pos[b] + r of sequence b from rows b * R + r of k_new, v_new (bf16 [n_seq * R][ld])
cudaError_t launch_kv_store(const KvBatch &c, const uint16_t *k_new, const uint16_t *v_new, int ld, int R,
                            const int64_t *pos, int *err, cudaStream_t s);
// the reverse: rows from entries (idle sequences' rows are zeros)
cudaError_t launch_kv_load(const KvBatch &c, const int64_t *pos, int R, uint16_t *k_out, uint16_t *v_out, int ld,
                           int *err, cudaStream_t s);

}  // namespace tfk
