// What the tcgen05 attention kernels share: tiles of 128 query vectors, the order of
// their K and V tiles, and small device helpers.
#pragma once
#include <cuda.h>

#include "kv_batch.cuh"
#include "tf_tcgen05.cuh"

namespace tfk {

constexpr float kScaleLog2 = 0.12751743074439720f;   // log2(e) / sqrt(128)
// A vector's reference maximum moves only when a score passes it by more than
// 2^8 in weight: weights stay below 2^8 (exact in the sums' exponents), and the
// output is rescaled rarely.  The decision is the vector's own.
constexpr float kMaxSlack = 8.0f / kScaleLog2;

constexpr int kTile = 128;              // query vectors and keys per matrix product
constexpr int kHalfBytes = kTile * 128; // 64 elements of 128 rows
constexpr int kTileBytes = 2 * kHalfBytes;

template <int N>
__device__ __forceinline__ void regs_raise() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_lower() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A bounded wait for what is still in flight when a role ends.
__device__ __forceinline__ void wait_drained(uint64_t *bar, uint32_t parity) {
    for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait(bar, parity); ++i) {
    }
}

// K and V tiles are taken in the order K0 K1 V0 K2 V1 ... V(n-1) of each item.
__device__ __forceinline__ int k_order(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int v_order(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }
// The tile at place t of that order: whether it is a V tile, and which.
__device__ __forceinline__ bool order_is_v(int t, int n) { return t == 2 * n - 1 || (t != 0 && t % 2 == 0); }
__device__ __forceinline__ int order_tile(int t, int n) {
    return t == 2 * n - 1 ? n - 1 : (t == 0 ? 0 : (t % 2 == 0 ? t / 2 - 1 : (t + 1) / 2));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 32 bytes, 32-byte aligned: a whole sector by one thread.
__device__ __forceinline__ void st_global_32(void *p, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ bool bf16x2_nonfinite(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
// The same as bits: the sum carries into kNonfiniteBits where a half's exponent is all ones, and the halves do not
// meet.  The other bits are anything.
constexpr uint32_t kNonfiniteBits = 0x80008000u;
__device__ __forceinline__ uint32_t bf16x2_nonfinite_bits(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t bf16x2_finite(uint32_t w) {   // non-finite halves -> 0
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
    return w;
}

// A weight e^(s - m) is above zero, however far it lies below what the sums hold, so an output whose column
// of V holds values that are not finite, among the entries that its vector attends over, is their sum: an infinity, or
// NaN.  A product gives that up to weights that are zero here (0 * inf is NaN), which depends on the rows
// beside a vector where an entry's value was taken out of a tile and added later.  So the kernels that write
// outputs look whether one is not finite where its weights' sum is (a product a pair of outputs with a zero), and then
// look through the entries of its column.  That is a rare and slow path: no tile is looked over for it.
__device__ __forceinline__ uint32_t probe_finite(uint32_t pair, uint32_t so_far) { return fma_bf16x2(pair, 0u, so_far); }
// x += the non-finite of a chunk's eight values, or of a quad's four
__device__ __forceinline__ void add_nonfinite(uint32_t w, float &x0, float &x1) {
    if ((w & 0x7F80u) == 0x7F80u) x0 += __uint_as_float(w << 16);
    if ((w & 0x7F800000u) == 0x7F800000u) x1 += __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void add_nonfinite(const uint4 &w, float (&x)[8]) {
    add_nonfinite(w.x, x[0], x[1]);
    add_nonfinite(w.y, x[2], x[3]);
    add_nonfinite(w.z, x[4], x[5]);
    add_nonfinite(w.w, x[6], x[7]);
}
// The sum of the non-finite values among a quad of columns (4 quad ..) of entries first .. last of one head's bf16 cache.
__device__ __noinline__ inline float4 cached_nonfinite(const uint16_t *v, int first, int last, int quad) {
    constexpr int kAtOnce = 8;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int t0 = first; t0 <= last; t0 += kAtOnce) {
        uint2 w[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {     // the last entry again changes nothing
            const int t = min(t0 + i, last);
            w[i] = *reinterpret_cast<const uint2 *>(v + (size_t)t * kHeadDim + 8 * ((quad >> 1) ^ (t & 7)) + 4 * (quad & 1));
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            add_nonfinite(w[i].x, x.x, x.y);
            add_nonfinite(w[i].y, x.z, x.w);
        }
    }
    return x;
}
__device__ __forceinline__ float4 add4(const float4 &x, const float4 &y) {
    return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
}
// The sum's non-zero elements take the place of four outputs.
__device__ __forceinline__ void put_nonfinite(uint16_t *out, const float4 &x) {
    if (x.x != 0.f) out[0] = __bfloat16_as_ushort(__float2bfloat16_rn(x.x));
    if (x.y != 0.f) out[1] = __bfloat16_as_ushort(__float2bfloat16_rn(x.y));
    if (x.z != 0.f) out[2] = __bfloat16_as_ushort(__float2bfloat16_rn(x.z));
    if (x.w != 0.f) out[3] = __bfloat16_as_ushort(__float2bfloat16_rn(x.w));
}

// Tiled map of bf16 elements, innermost dimension first (its stride is 1; strides in
// bytes); false and *why where there is none.
template <int N>
bool encode_tiles(CUtensorMap *m, const void *base, const cuuint64_t (&dims)[N], const cuuint64_t (&strides)[N - 1],
                  const cuuint32_t (&box)[N], CUtensorMapSwizzle swizzle, const char **why);

}  // namespace tfk
