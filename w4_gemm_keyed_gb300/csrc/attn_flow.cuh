// The flow of causal attention through one CTA, which the kernels for whole prompts and
// for trees of drafts share: tiles of 128 query vectors (whole rows of one KV head's
// query heads), two of them to an item, and the item's keys kKeys at a time.
//
// S = Q K^T with both operands in shared memory and S in tensor memory; a thread per vector
// turns S into weights P (bf16, tensor memory) with a running maximum; O += P V with P read from
// tensor memory.  Keys are taken 80 at a time because tensor memory (512 columns) then holds,
// next to two tiles' outputs (256), their scores (160) and their weights (80) apart: the next
// scores are computed while this step's weights are formed, and the products never wait for the
// chain scores - softmax - weights of one step.
//
// Roles: softmax in warps 0-7 (four a tile; items of one tile leave the other four idle), a thread each
// that issues scores and outputs, a warp that mends V tiles, and the kernel's own:
// a producer of items, queries, K and V tiles, and who stores the outputs.
#pragma once
#include <cuda_bf16.h>

#include "attn_tiles.cuh"

namespace tfk {
namespace flow {

constexpr int kKeys = 80;               // keys of a K or V tile
constexpr int kKeyHalf = kKeys * 128;   // 64 elements of a tile's rows
constexpr int kKeyBytes = 2 * kKeyHalf;
constexpr int kRing = 4;                // items known ahead
constexpr int kMends = 4;               // V tiles to mend on their way: at most their stages, and an end mark
constexpr int kSoftmaxWarps = 8;
constexpr uint32_t kTmemCols = 512, kTmemO = 0, kTmemS = 256, kTmemP = kTmemS + 2 * kKeys;
constexpr uint32_t kPStride = (kKeys / 2 + 15) / 16 * 16;      // columns of a tile's weights
static_assert(kTmemP + 2 * kPStride <= kTmemCols, "tensor memory");
static_assert(kKeyHalf % 1024 == 0 && kKeys % 16 == 0, "whole swizzle atoms and product steps");

// What the common roles need of an item; a kernel's own adds to it.
struct ItemBase {
    int n_rows;         // rows of the item (0: no more items)
    int n_keys;         // its keys
};

struct Mend {
    int stage;          // of the V tile; -1: no more
    int slot;           // of its item in the ring
    int first, valid;   // first row that some vector of the item does not see; rows of the sequence in the tile
};

// A parity wait tells a phase from its neighbours only, so whoever waits on a
// barrier waits on every one of its phases, and before the next can end.  Index: tile of an item.
template <typename ITEM, int K_STAGES, int V_STAGES, int QUERIES>
struct __align__(16) SharedBase {
    static constexpr int k_stages = K_STAGES, v_stages = V_STAGES, queries = QUERIES;
    static_assert(V_STAGES < kMends, "room for the end mark");
    uint64_t k_full[K_STAGES], k_empty[K_STAGES], v_full[V_STAGES], v_empty[V_STAGES], mend_full[kMends];
    uint64_t q_full[QUERIES], q_empty[QUERIES];
    uint64_t s_full[2], s_free[2], p_full[2], o_done[2];
    uint64_t o_last[2], o_free[2];      // a tile's last product of an item; its output taken
    uint64_t item_full[kRing], item_empty[kRing], drain[2];
    ITEM item[kRing];
    Mend mend[kMends];
    int bad[kRing];     // whether a value that only some vectors see is not finite
    uint32_t tmem;
    int abort;

    // One thread, before the roles start.  tile_arrivals: on a K or V tile (copies, or the warps that
    // expand it); readers: warps and threads that take items; storers: warps that take a tile's output.
    __device__ void init(int tile_arrivals, int readers, int storers) {
        for (int i = 0; i < K_STAGES; ++i) {
            mbar_init(&k_full[i], tile_arrivals);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < V_STAGES; ++i) {
            mbar_init(&v_full[i], tile_arrivals);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kMends; ++i) mbar_init(&mend_full[i], 1);
        for (int i = 0; i < QUERIES; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 4);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
            mbar_init(&o_last[i], 1);
            mbar_init(&o_free[i], storers);
            mbar_init(&drain[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], readers);
        }
        abort = 0;
    }
};

// A wait of one thread that is its warp's only one in the role.
template <typename SHARED>
__device__ __forceinline__ bool lane_wait(SHARED *sh, uint64_t *bar, uint32_t parity) {
    return mbar_wait_or_abort(&sh->abort, bar, parity);
}
// A wait of a converged warp: all lanes get one answer.
template <typename SHARED>
__device__ __forceinline__ bool warp_wait(SHARED *sh, uint64_t *bar, uint32_t parity) {
    return mbar_warp_wait_or_abort(&sh->abort, bar, parity);
}

// The same of roles that mostly wait: less code, and a few cycles more where the phase is already over.
template <typename SHARED>
__device__ __forceinline__ bool lane_idle_wait(SHARED *sh, uint64_t *bar, uint32_t parity) {
#pragma unroll 1
    for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i) {
        if (i == kWaitLimit) *reinterpret_cast<volatile int *>(&sh->abort) = 1;
        if (*reinterpret_cast<volatile int *>(&sh->abort)) return false;
    }
    return true;
}
template <typename SHARED>
__device__ __forceinline__ bool warp_idle_wait(SHARED *sh, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, lane_idle_wait(sh, bar, parity));
}

// A tile of queries is whole rows of a KV head's query heads, a box of (64 elements, heads, rows, halves): both halves in one copy
// where they are 128 vectors, whose halves then lie where the products expect them.  Rows of the box past the
// item's fill vectors that nothing reads: rows of a product never mix.  One thread.
__device__ __forceinline__ void load_queries(uint8_t *dst, const CUtensorMap *map, int head, int row, int vectors, uint64_t *bar) {
    mbar_arrive_expect_tx(bar, 2 * uint32_t(vectors) * 128u);
    tma_load_4d(dst, map, 0, head, row, 0, bar);
    if (vectors < kTile) tma_load_4d(dst + kHalfBytes, map, 0, head, row, 1, bar);
}
inline bool encode_queries(CUtensorMap *m, const uint16_t *base, int heads, int rows, int ld, int group, int rows_tile, const char **why) {
    return encode_tiles<4>(m, base, {64, cuuint64_t(heads), cuuint64_t(rows), 2}, {cuuint64_t(kHeadDim) * 2, cuuint64_t(ld) * 2, 128},
                           {64, cuuint32_t(group), cuuint32_t(rows_tile), group * rows_tile == kTile ? 2u : 1u},
                           CU_TENSOR_MAP_SWIZZLE_128B, why);
}

// A place in a ring of N barriers, and the parity of the phase that is awaited there.
template <int N>
struct Ring {
    int at = 0;
    uint32_t parity = 0;
    __device__ void step() {
        if (++at == N) {
            at = 0;
            parity ^= 1u;
        }
    }
};

// V tiles that hold rows some vectors of the item do not see: rows past the item's
// last become zeros (up to the 16-row step the product reads; they are another sequence's,
// or nobody's), and non-finite elements of rows that only some vectors see become zero, since
// 0 * inf would reach the others; the vectors that see them get them back when
// the output is stored (attn_tiles.cuh).
template <typename SHARED>
__device__ void mend_tiles(SHARED *sh, uint8_t *v_tiles) {
    const int lane = threadIdx.x & 31, c = lane & 15;
    constexpr int kAtOnce = 4;          // pairs of rows
    for (unsigned n = 0;; ++n) {
        const int slot = n % kMends;
        if (!warp_idle_wait(sh, &sh->mend_full[slot], (n / kMends) & 1)) return;
        const Mend m = sh->mend[slot];
        if (m.stage < 0) return;
        uint8_t *v = v_tiles + size_t(m.stage) * kKeyBytes + (c >> 3) * kKeyHalf;
        auto at = [&](int row) { return reinterpret_cast<uint4 *>(v + row * 128 + (((c & 7) ^ (row & 7)) << 4)); };
        const int end = (m.valid + 15) & ~15;
        // Nearly always there is nothing to mend, and the outputs wait for knowing it.
        uint32_t found = 0u;
#pragma unroll 1
        for (int row0 = m.first + (lane >> 4); row0 < m.valid; row0 += 2 * kAtOnce) {
            uint4 x[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                x[i] = *at(min(row0 + 2 * i, m.valid - 1));
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                found |= bf16x2_nonfinite_bits(x[i].x) | bf16x2_nonfinite_bits(x[i].y) | bf16x2_nonfinite_bits(x[i].z) |
                         bf16x2_nonfinite_bits(x[i].w);
        }
        if (found & kNonfiniteBits) {
#pragma unroll 1
            for (int row = m.first + (lane >> 4); row < m.valid; row += 2) {
                const uint4 x = *at(row);
                *at(row) = make_uint4(bf16x2_finite(x.x), bf16x2_finite(x.y), bf16x2_finite(x.z), bf16x2_finite(x.w));
            }
            *reinterpret_cast<volatile int *>(&sh->bad[m.slot]) = 1;
        }
#pragma unroll 1
        for (int row = m.valid + (lane >> 4); row < end; row += 2) *at(row) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->v_full[m.stage]);
    }
}

// The items in order, for a role of one thread; what it needs of one.
template <typename SHARED>
struct Items {
    SHARED *sh;
    int rows_tile;
    Ring<kRing> ring;
    int tiles = 0, n_keys = 0;
    bool two = false;
    __device__ bool next() {        // false: no more, or gave up
        if (!lane_idle_wait(sh, &sh->item_full[ring.at], ring.parity)) return false;
        const ItemBase it = sh->item[ring.at];
        mbar_arrive(&sh->item_empty[ring.at]);
        ring.step();
        two = it.n_rows > rows_tile;
        n_keys = it.n_keys;
        tiles = (n_keys + kKeys - 1) / kKeys;
        return it.n_rows != 0;
    }
    __device__ int steps16(int i) const { return (min(kKeys, n_keys - i * kKeys) + 15) >> 4; }
};

// Scores and outputs are issued by two threads, each of which waits for what its own
// products need: every wait and commit costs the thread that issues them some 100 cycles,
// and one thread for both took 2,600 cycles a step of two tiles where the products take 1,450.

// S[t] = Q[t] K(i)^T for the item's one or two tiles t, key tile by key tile (rounded up to 16 keys).
template <typename SHARED>
__device__ void issue_scores(SHARED *sh, int rows_tile, const uint8_t *q_tiles, const uint8_t *k_tiles, uint32_t tmem) {
    Items<SHARED> items{sh, rows_tile};
    Ring<SHARED::k_stages> tile;
    Ring<SHARED::queries> query;
    uint32_t free_parity[2] = {1u, 1u};     // of a fresh barrier, the phase before the first counts as over
    const uint32_t q_addr = smem_u32(q_tiles), k_addr = smem_u32(k_tiles);
    bool ok = true;
    while (ok && items.next()) {
        uint32_t a[2] = {0u, 0u};
        uint64_t *done[2] = {nullptr, nullptr};
        const int last = items.tiles - 1;
        for (int i = 0; i <= last && ok; ++i) {
            const uint32_t idesc = umma_idesc_bf16(kTile, 16 * items.steps16(i), false);
            const uint32_t b = umma_desc_low(k_addr + tile.at * kKeyBytes, 16);
            ok = lane_wait(sh, &sh->k_full[tile.at], tile.parity);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (t == 1 && !items.two) break;
                if (i == 0) {
                    ok = ok && lane_wait(sh, &sh->q_full[query.at], query.parity);
                    a[t] = umma_desc_low(q_addr + query.at * kTileBytes, 16);
                    done[t] = &sh->q_empty[query.at];
                    query.step();
                }
                ok = ok && lane_wait(sh, &sh->s_free[t], free_parity[t]);
                if (!ok) break;
                free_parity[t] ^= 1u;
                tc_fence_after();
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    tc_mma_ss(tmem + kTmemS + t * kKeys, a[t] + (((d >> 2) * kHalfBytes + (d & 3) * 32) >> 4),
                              b + (((d >> 2) * kKeyHalf + (d & 3) * 32) >> 4), idesc, d > 0);
                tc_commit(&sh->s_full[t]);
                if (i == last) tc_commit(done[t]);
            }
            tc_commit(&sh->k_empty[tile.at]);
            tile.step();
        }
    }
    // no product outlives the CTA, whichever way the loop ended
    tc_commit(&sh->drain[0]);
    wait_drained(&sh->drain[0], 0);
}

// O[t] (+)= P[t] V(i) likewise.
template <typename SHARED>
__device__ void issue_outputs(SHARED *sh, int rows_tile, const uint8_t *v_tiles, uint32_t tmem) {
    Items<SHARED> items{sh, rows_tile};
    Ring<SHARED::v_stages> tile;
    uint32_t p_parity[2] = {0u, 0u}, free_parity[2] = {1u, 1u};
    const uint32_t v_addr = smem_u32(v_tiles);
    constexpr uint32_t idesc = umma_idesc_bf16(kTile, kHeadDim, true);
    bool ok = true;
    while (ok && items.next()) {
        const int last = items.tiles - 1;
        for (int i = 0; i <= last && ok; ++i) {
            const int steps = items.steps16(i);
            const uint32_t b = umma_desc_low(v_addr + tile.at * kKeyBytes, kKeyHalf);
            ok = lane_wait(sh, &sh->v_full[tile.at], tile.parity);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (t == 1 && !items.two) break;
                const uint32_t d = tmem + kTmemO + t * kHeadDim, a = tmem + kTmemP + t * kPStride;
                ok = ok && lane_wait(sh, &sh->p_full[t], p_parity[t]);
                if (i == 0) {       // the last item's output has been taken
                    ok = ok && lane_wait(sh, &sh->o_free[t], free_parity[t]);
                    free_parity[t] ^= 1u;
                }
                if (!ok) break;
                p_parity[t] ^= 1u;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < kKeys / 16; ++s)
                    if (s < steps) tc_mma_ts(d, a + 8 * s, b + s * 128, idesc, i > 0 || s > 0);
                tc_commit(&sh->o_done[t]);
                if (i == last) tc_commit(&sh->o_last[t]);
            }
            tc_commit(&sh->v_empty[tile.at]);
            tile.step();
        }
    }
    tc_commit(&sh->drain[1]);
    wait_drained(&sh->drain[1], 0);
}

// Two scores to two weights, added to the sums.  Weights meet V as bf16 (off by at
// most 2^-8 of each, half a step); the sums keep them whole.
__device__ __forceinline__ uint32_t weigh(uint32_t s0, uint32_t s1, uint64_t scale2, uint64_t shift2, uint64_t &sum2) {
    float a, b;
    unpack2(fma2(pack2(__uint_as_float(s0), __uint_as_float(s1)), scale2, shift2), a, b);
    a = ex2_approx(a);
    b = ex2_approx(b);
    sum2 = add2(sum2, pack2(a, b));
    const __nv_bfloat162 pk = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&pk);
}

// What the vectors of a warp see of an item's keys: this thread's last, and the least and greatest of the warp.
struct Sight {
    int last, least, greatest;
};

// sight(slot of the item, item, tile, rows of the tile, this thread's row and the warp's first and last in
// the tile), and at the item's end finish(slot, tile, rows of the tile, this thread's maximum and sum, steps of the tile so far), false
// where a wait gave up: whole warp.  KEEP: the item stays in its slot until then.
template <bool KEEP, typename SHARED, typename SIGHT, typename FINISH>
__device__ void softmax(SHARED *sh, int rows_tile, int group, uint32_t tmem, SIGHT sight, FINISH finish) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wg = warp >> 2;
    const uint32_t my_lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t t_o = tmem + kTmemO + wg * kHeadDim + my_lanes, t_s = tmem + kTmemS + wg * kKeys + my_lanes,
                   t_p = tmem + kTmemP + wg * kPStride + my_lanes;
    const int v0 = 32 * (warp & 3), row_first = v0 / group, row_last = (v0 + 31) / group,
              my_row = (v0 + lane) / group;
    const uint64_t scale2 = pack2(kScaleLog2, kScaleLog2);
    unsigned steps = 0;     // of this group
    auto hand = [&](uint64_t *bar) {        // what the warp has read or written in tensor memory
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (!warp_wait(sh, &sh->item_full[slot], (n / kRing) & 1)) return;
        const int n_rows = sh->item[slot].n_rows, n_keys = sh->item[slot].n_keys;
        const int n_here = min(rows_tile, n_rows - wg * rows_tile);     // rows of this tile
        const Sight see = n_here > 0 ? sight(slot, sh->item[slot], wg, n_here, my_row, row_first, row_last) : Sight{};
        auto release = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
        };
        if (!KEEP || n_here <= 0) release();
        if (n_rows == 0) return;
        if (n_here <= 0) continue;
        const int tiles = (n_keys + kKeys - 1) / kKeys, lim = see.last;
        const bool active = row_first < n_here;
        float m = -INFINITY, l = 0.f;
        bool done;      // whether the step before is known to have used its weights and left its part of the output
        auto wait_done = [&] {
            const bool ok = done || warp_wait(sh, &sh->o_done[wg], (steps - 1) & 1);
            done = true;
            tc_fence_after();
            return ok;
        };
        // The running maximum takes in this step's, and the outputs so far are rescaled if
        // it moves; false where a wait gave up.
        auto fold = [&](float top, bool first, uint64_t &shift2) {
            const bool moved = top > m + kMaxSlack;     // true for the first visible scores (m = -inf)
            float scale = 1.f;
            if (moved) {
                scale = ex2_approx((m - top) * kScaleLog2);
                m = top;
                l *= scale;
            }
            if (!first && __any_sync(0xFFFFFFFFu, moved)) {
                if (!wait_done()) return false;
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t o[16];
                    tc_ld16(t_o + 16 * c, o);
                    tc_wait_ld();
                    tc_pin16(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
                    tc_st16(t_o + 16 * c, o);
                }
                tc_wait_st();
            }
            const float mc = m == -INFINITY ? 0.f : m * kScaleLog2;
            shift2 = pack2(-mc, -mc);
            return true;
        };
        for (int i = 0; i < tiles; ++i, ++steps) {
            if (!warp_wait(sh, &sh->s_full[wg], steps & 1)) return;
            tc_fence_after();
            done = steps == 0;
            uint64_t sum2[2] = {0ull, 0ull}, shift2;
            if (!active) {
                hand(&sh->s_free[wg]);
                if (!wait_done()) return;
            } else if (see.least >= (i + 1) * kKeys - 1) {       // every vector sees every key
                uint32_t x[kKeys];
                tc_ld32(t_s, x);
                tc_ld32(t_s + 32, x + 32);
                tc_ld16(t_s + 64, x + 64);
                tc_wait_ld();
                tc_pin32(x);
                tc_pin32(x + 32);
                tc_pin16(x + 64);
                hand(&sh->s_free[wg]);
                float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kKeys; c += 2)
                    mt[(c >> 1) & 3] = max3(mt[(c >> 1) & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
                if (!fold(fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3])), i == 0, shift2)) return;
                // all weights before the wait: the last step's products go on meanwhile
#pragma unroll
                for (int c = 0; c < kKeys / 2; ++c) x[c] = weigh(x[2 * c], x[2 * c + 1], scale2, shift2, sum2[c & 1]);
                if (!wait_done()) return;
                tc_st32(t_p, x);
                tc_st8(t_p + 32, x + 32);
            } else {
                // 16 keys at a time, twice: as many as any vector of the warp sees
                const int key = i * kKeys, steps16 = (min(kKeys, n_keys - key) + 15) >> 4;
                const int seen = see.greatest < key ? 0 : min(steps16, ((see.greatest - key) >> 4) + 1);
                auto fetch = [&](int c, uint32_t *x) {
                    tc_ld16(t_s + 16 * c, x);
                    tc_wait_ld();
                    tc_pin16(x);
                    const int last = lim - key - 16 * c;
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = e <= last ? x[e] : 0xFF800000u;
                };
                float top = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < seen; ++c) {
                    uint32_t x[16];
                    fetch(c, x);
#pragma unroll
                    for (int e = 0; e < 16; e += 2) top = max3(top, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                }
                if (!fold(top, i == 0, shift2) || !wait_done()) return;
#pragma unroll 1
                for (int c = 0; c < steps16; ++c) {
                    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                    if (c < seen) {
                        uint32_t x[16];
                        fetch(c, x);
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = weigh(x[2 * e], x[2 * e + 1], scale2, shift2, sum2[e & 1]);
                    }
                    tc_st8(t_p + 8 * c, w);
                }
                hand(&sh->s_free[wg]);
            }
            tc_wait_st();
            float s0, s1, s2, s3;
            unpack2(sum2[0], s0, s1);
            unpack2(sum2[1], s2, s3);
            l += (s0 + s1) + (s2 + s3);
            if (!KEEP && i + 1 == tiles && !finish(slot, wg, n_here, m, l, steps)) return;
            hand(&sh->p_full[wg]);
        }
        if (KEEP) {
            if (!finish(slot, wg, n_here, m, l, steps)) return;
            release();
        }
    }
}

}  // namespace flow
}  // namespace tfk
