// Causal attention of whole prompts, packed one after the other.
//
// Row i of a sequence attends over its rows 0 .. i:
//   s_t = q . k_t / sqrt(128),  o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m).
//
// A tile is 128 query vectors: whole rows of one KV head's query heads (a vector is a
// row and a head), so that a K and V tile in shared memory serves every head that reads it
// and short prompts fill their tiles.  An item is two neighbouring tiles (one where
// there are few); each vector folds the keys of its sequence in ascending order,
// 128 at a time from the sequence's first row, with a running maximum, and no other vector's
// values ever mix with its own: its bits depend on its own query and keys alone.
// Scores and outputs run on tcgen05: S = Q K^T with both operands in shared memory
// and S in tensor memory, then P (bf16, in place of S) times V with P read from tensor
// memory.  Persistent CTAs take items from a counter, the longest first over all sequences.
#include <atomic>

#include <cuda_bf16.h>

#include "attn_prompt.cuh"
#include "attn_tiles.cuh"
#include "w4_gemm.cuh"

namespace tfk {

namespace {

constexpr int kStages = 5;              // K and V tiles in shared memory
constexpr int kRing = 4;                // items known ahead
constexpr int kMends = 8;               // V tiles to mend on their way: at most kStages, and two end marks
constexpr int kSoftmaxWarps = 8, kProducerWarp = 8, kMmaWarp = 9, kMendWarp = 10, kMendWarps = 2;
constexpr int kCtaThreads = 384;
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
static_assert(256 * kRegsSoftmax + (kCtaThreads - 256) * kRegsOther <= kCtaThreads * 168, "register split");
constexpr int kReaders = kSoftmaxWarps + 1;     // of the item ring
constexpr uint32_t kTmemCols = 512, kTmemS = 0, kTmemO = 256;

struct Item {
    int n_rows;         // rows of the item (0: no more items)
    int j;              // KV head
    int i0;             // first row's place in its sequence
    int seq0;           // the sequence's first row in the arrays
};

struct Mend {
    int stage;          // of the V tile; -1: no more
    int slot;           // of its item in the ring
    int first, valid;   // first row that some vector of the item does not see; rows of the sequence in the tile
};

struct KernelArgs {
    CUtensorMap q, k, v;
    AttnPromptArgs a;
    int rows_tile;      // rows per tile of 128 vectors
    int rows_item;      // rows per item: one or two tiles
    unsigned *next;     // items taken beyond the first of each CTA, and CTAs done; both zero between calls
};

// A parity wait tells a phase from its neighbours only, so whoever waits on a
// barrier waits on every one of its phases, and before the next can end.  Hence three barriers for scores:
// S0 and S1 of one-tile items and S0 of two-tile items are read by the first
// softmax group (0, 1, 0), S1 of two-tile items by the second (2).
struct __align__(16) Shared {
    uint64_t kv_full[kStages], kv_empty[kStages], mend_full[kMends];
    uint64_t q_full[2], q_empty[2], s_full[3], p_full[2][2], o_done[2];
    uint64_t item_full[kRing], item_empty[kRing], drain;
    Item item[kRing];
    Mend mend[kMends];
    int bad[kRing];     // whether a value that only some vectors see is not finite
    uint32_t tmem;
    int abort;
};
constexpr size_t kSmemBytes = size_t(2 + kStages) * kTileBytes + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// A wait of one thread that is its warp's only one in the role.
__device__ __forceinline__ bool lane_wait(Shared *sh, uint64_t *bar, uint32_t parity) {
    return mbar_wait_or_abort(&sh->abort, bar, parity);
}
// A wait of a converged warp: all lanes get one answer.
__device__ __forceinline__ bool warp_wait(Shared *sh, uint64_t *bar, uint32_t parity) {
    return mbar_warp_wait_or_abort(&sh->abort, bar, parity);
}

// ------------------------------------------------------------------ item order
// Items in descending order of their place in their sequences (so of their cost):
// level by level, at each level the sequences that reach it, heads fastest.  The set
// of sequences that reach a level changes only where one of them ends, so a whole run of levels is
// found with one pass over the sequences.  A warp's work, in step.
struct Finder {
    const KernelArgs &k;
    int next_level, high, count;
    unsigned first, end;

    __device__ int levels(int s) const {    // items of sequence s and head
        return int(idx_div(unsigned(k.a.starts[s + 1] - k.a.starts[s]) + k.rows_item - 1, k.rows_item));
    }
    // Whole warp.  Starts that fall or lie outside the rows: no items.
    __device__ explicit Finder(const KernelArgs &args) : k(args), next_level(-1), high(0), count(0), first(0), end(0) {
        const int lane = threadIdx.x & 31;
        bool bad = false;
        int top = 0;
        for (int s = lane; s < k.a.n_seq; s += 32) {
            const long long x = k.a.starts[s], y = k.a.starts[s + 1];
            if (x < 0 || y < x || y > k.a.rows)
                bad = true;
            else
                top = max(top, levels(s));
        }
        if (__any_sync(0xFFFFFFFFu, bad)) {
            if (blockIdx.x == 0 && lane == 0) set_error(k.a.err, kDevBadPosition);
            return;
        }
        next_level = __reduce_max_sync(0xFFFFFFFFu, top) - 1;
    }
    // Whole warp; i never falls from call to call.
    __device__ Item find(unsigned i) {
        const int lane = threadIdx.x & 31;
        Item it{};
        while (i >= end) {
            if (next_level < 0) return it;
            int more = 0, below = 0;
            for (int s = lane; s < k.a.n_seq; s += 32) {
                const int n = levels(s);
                if (n > next_level)
                    ++more;
                else
                    below = max(below, n);
            }
            count = __reduce_add_sync(0xFFFFFFFFu, more);
            below = __reduce_max_sync(0xFFFFFFFFu, below);
            first = end;
            end += unsigned(next_level - below + 1) * unsigned(count) * unsigned(k.a.n_kv);
            high = next_level;
            next_level = below - 1;
        }
        const unsigned per_level = unsigned(count) * unsigned(k.a.n_kv), off = i - first;
        const int level = high - int(off / per_level);
        const unsigned rest = off % per_level;
        int nth = int(rest / unsigned(k.a.n_kv));
        it.j = int(rest % unsigned(k.a.n_kv));
        for (int s0 = 0;; s0 += 32) {       // the nth sequence that reaches the level: there is one
            const int s = s0 + lane;
            const unsigned reach = __ballot_sync(0xFFFFFFFFu, s < k.a.n_seq && levels(s) > high);
            const int here = __popc(reach);
            if (nth < here) {
                const int at = s0 + __fns(reach, 0, nth + 1);
                it.seq0 = int(k.a.starts[at]);
                it.i0 = level * k.rows_item;
                it.n_rows = min(k.rows_item, int(k.a.starts[at + 1]) - it.seq0 - it.i0);
                return it;
            }
            nth -= here;
            if (s0 >= k.a.n_seq) return Item{};     // not reached
        }
    }
};

// ------------------------------------------------------------------ roles
//   warp 8      finds the next item and streams its query vectors and its K and V
//               tiles by TMA
//   warp 9      issues the products
//   warps 10-11 mend V tiles that reach past what all the item's vectors see
//   warps 0-7   softmax: a thread per vector.  Items of two tiles give one tile to
//               each group of four warps; items of one tile use the second tile's
//               S columns so that the next key tile's scores are computed
//               while this one's are being exponentiated.

__device__ void produce(const KernelArgs &k, Shared *sh, uint8_t *q_tiles, uint8_t *stages) {
    const int lane = threadIdx.x & 31;
    Finder finder(k);
    unsigned i = blockIdx.x;
    unsigned loaded = 0;            // K and V tiles so far
    unsigned mended = 0;            // of them V tiles to mend
    unsigned to_mend = 0;           // bit st: the last tile of stage st is one
    unsigned q_uses[2] = {0, 0};
    int q_next = 0;                 // the query tile of the next one-tile item
    const int g = k.a.group;
    bool ok = true;
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (n >= kRing && !warp_wait(sh, &sh->item_empty[slot], (n / kRing - 1) & 1)) break;
        const Item it = finder.find(i);
        unsigned taken = 0;
        if (lane == 0) {
            sh->item[slot] = it;
            sh->bad[slot] = 0;
            mbar_arrive(&sh->item_full[slot]);
            if (it.n_rows) taken = atomicAdd(k.next, 1u);       // the item after this one
        }
        if (it.n_rows == 0) break;
        if (lane == 0) {
            const int n_keys = it.i0 + it.n_rows, tiles = (n_keys + kTile - 1) / kTile;
            // A tile of queries is whole rows of the KV head's query heads, one box of (64
            // elements, heads, rows) per half.  Rows of the box past the item's
            // fill vectors that nothing reads: rows of a product never mix.
            const bool two = it.n_rows > k.rows_tile;
            for (int t = 0; t < (two ? 2 : 1) && ok; ++t) {
                const int buf = two ? t : q_next;
                if (q_uses[buf] > 0) ok = lane_wait(sh, &sh->q_empty[buf], (q_uses[buf] - 1) & 1);
                if (!ok) break;
                ++q_uses[buf];
                const int row = it.seq0 + it.i0 + t * k.rows_tile;
                mbar_arrive_expect_tx(&sh->q_full[buf], 2 * uint32_t(k.rows_tile * g) * 128u);
                tma_load_3d(q_tiles + buf * kTileBytes, &k.q, 0, it.j * g, row, &sh->q_full[buf]);
                tma_load_3d(q_tiles + buf * kTileBytes + kHalfBytes, &k.q, 64, it.j * g, row, &sh->q_full[buf]);
            }
            if (!two) q_next ^= 1;
            for (int t = 0; t < 2 * tiles && ok; ++t, ++loaded) {
                const bool is_v = order_is_v(t, tiles);
                const int key = order_tile(t, tiles) * kTile, st = loaded % kStages;
                if (loaded >= kStages) ok = lane_wait(sh, &sh->kv_empty[st], (loaded / kStages - 1) & 1);
                if (!ok) break;
                uint64_t *bar = &sh->kv_full[st];
                const int first = max(0, it.i0 + 1 - key);
                to_mend &= ~(1u << st);
                if (is_v && first < kTile) {        // past the first row's last key: handed over by its mender
                    const int m = mended++ % kMends;
                    sh->mend[m] = {st, slot, first, min(kTile, n_keys - key)};
                    to_mend |= 1u << st;
                    bar = &sh->mend_full[m];
                }
                uint8_t *dst = stages + size_t(st) * kTileBytes;
                mbar_arrive_expect_tx(bar, kTileBytes);
                tma_load_3d(dst, is_v ? &k.v : &k.k, 0, it.j, it.seq0 + key, bar);
                tma_load_3d(dst + kHalfBytes, is_v ? &k.v : &k.k, 64, it.j, it.seq0 + key, bar);
            }
        }
        __syncwarp();
        if (!__shfl_sync(0xFFFFFFFFu, int(ok), 0)) break;
        i = gridDim.x + __shfl_sync(0xFFFFFFFFu, taken, 0);
    }
    if (lane != 0) return;
    // no copy outlives the CTA
    for (unsigned t = loaded > kStages ? loaded - kStages : 0; t < loaded; ++t)
        if (!(to_mend >> (t % kStages) & 1u)) wait_drained(&sh->kv_full[t % kStages], (t / kStages) & 1);
    for (unsigned t = mended > kStages ? mended - kStages : 0; t < mended; ++t)
        wait_drained(&sh->mend_full[t % kMends], (t / kMends) & 1);
    for (int buf = 0; buf < 2; ++buf)
        if (q_uses[buf] > 0) wait_drained(&sh->q_full[buf], (q_uses[buf] - 1) & 1);
    for (int w = 0; w < kMendWarps; ++w, ++mended) {
        sh->mend[mended % kMends].stage = -1;
        mbar_arrive(&sh->mend_full[mended % kMends]);
    }
}

// V tiles that hold rows some vectors of the item do not see: rows past the item's
// last become zeros (up to the 16-row step the product reads; they are another sequence's,
// or nobody's), and non-finite elements of rows that only some vectors see become zero, since
// 0 * inf would reach the others; the vectors that see them get them back when
// the output is stored.  The two warps take such tiles in turn.
__device__ void mend_tiles(Shared *sh, uint8_t *stages) {
    const int lane = threadIdx.x & 31;
    for (unsigned n = (threadIdx.x >> 5) - kMendWarp;; n += kMendWarps) {
        const int slot = n % kMends;
        if (!warp_wait(sh, &sh->mend_full[slot], (n / kMends) & 1)) return;
        const Mend m = sh->mend[slot];
        if (m.stage < 0) return;
        uint8_t *v = stages + size_t(m.stage) * kTileBytes;
        const int end = (m.valid + 15) & ~15;
        bool bad = false;
        for (int i = m.first * 16 + lane; i < end * 16; i += 32) {
            const int row = i >> 4, c = i & 15;
            uint4 *p = reinterpret_cast<uint4 *>(v + (c >> 3) * kHalfBytes + row * 128 + (((c & 7) ^ (row & 7)) << 4));
            if (row >= m.valid) {
                *p = make_uint4(0u, 0u, 0u, 0u);
            } else {
                const uint4 x = *p;
                if (bf16x2_nonfinite(x.x) || bf16x2_nonfinite(x.y) || bf16x2_nonfinite(x.z) || bf16x2_nonfinite(x.w)) {
                    *p = make_uint4(bf16x2_finite(x.x), bf16x2_finite(x.y), bf16x2_finite(x.z), bf16x2_finite(x.w));
                    bad = true;
                }
            }
        }
        if (bad) *reinterpret_cast<volatile int *>(&sh->bad[m.slot]) = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->kv_full[m.stage]);
    }
}

// The whole warp follows the items; the elected lane waits, issues and commits.
__device__ void multiply(const KernelArgs &k, Shared *sh, uint8_t *q_tiles, uint8_t *stages, uint32_t tmem) {
    const int lane = threadIdx.x & 31;
    const bool leader = elect_one() != 0;
    unsigned before = 0;                 // K and V tiles of the items before this one
    unsigned q_uses[2] = {0, 0}, p_uses[2] = {0, 0};
    int next = 0;
    const uint32_t q_addr = smem_u32(q_tiles), st_addr = smem_u32(stages);

    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (!warp_wait(sh, &sh->item_full[slot], (n / kRing) & 1)) break;
        // broadcast: the same in all lanes, and known to be
        const int n_rows = __shfl_sync(0xFFFFFFFFu, sh->item[slot].n_rows, 0);
        const int n_keys = __shfl_sync(0xFFFFFFFFu, sh->item[slot].i0, 0) + n_rows;
        if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
        __syncwarp();
        if (n_rows == 0) break;
        const bool two = n_rows > k.rows_tile;
        const int tiles = (n_keys + kTile - 1) / kTile;
        const int q0 = two ? 0 : next;
        auto stage_of = [&](int order) { return (before + order) % kStages; };
        auto wait_tile = [&](int order) {
            return lane_wait(sh, &sh->kv_full[stage_of(order)], ((before + order) / kStages) & 1);
        };
        // S[s] = Q[qb] K(i)^T over the keys of tile i (rounded up to 16)
        auto scores = [&](int qb, int s, int i) {
            const int keys = min(kTile, n_keys - i * kTile);
            const uint32_t idesc = umma_idesc_bf16(kTile, (keys + 15) & ~15, false);
            const uint32_t a = umma_desc_low(q_addr + qb * kTileBytes, 16);
            const uint32_t b = umma_desc_low(st_addr + stage_of(k_order(i)) * kTileBytes, 16);
            tc_fence_after();
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const uint32_t off = ((d >> 2) * kHalfBytes + (d & 3) * 32) >> 4;
                tc_mma_ss(tmem + kTmemS + s * kTile, a + off, b + off, idesc, d > 0);
            }
            tc_commit(&sh->s_full[two && s ? 2 : s]);
        };
        // O[o] (+)= P[s] V(i), 64 keys at a time as their weights arrive (the first have)
        auto outputs = [&](int o, int s, int i) {
            const int steps = (min(kTile, n_keys - i * kTile) + 15) >> 4;
            const uint32_t idesc = umma_idesc_bf16(kTile, kHeadDim, true);
            const uint32_t b = umma_desc_low(st_addr + stage_of(v_order(i, tiles)) * kTileBytes, kHalfBytes);
            const uint32_t d = tmem + kTmemO + o * kHeadDim, a = tmem + kTmemS + s * kTile;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1 && !lane_wait(sh, &sh->p_full[s][1], p_uses[s] & 1)) return false;
                tc_fence_after();
                if (steps >= 4 * h + 4) {
#pragma unroll
                    for (int t = 4 * h; t < 4 * h + 4; ++t) tc_mma_ts(d, a + 8 * t, b + t * 128, idesc, i > 0 || t > 0);
                } else {
                    for (int t = 4 * h; t < steps; ++t) tc_mma_ts(d, a + 8 * t, b + t * 128, idesc, i > 0 || t > 0);
                }
            }
            ++p_uses[s];
            tc_commit(&sh->o_done[o]);
            return true;
        };
        auto wait_probs = [&](int s) {      // the first 64 keys' weights
            return lane_wait(sh, &sh->p_full[s][0], p_uses[s] & 1);
        };
        auto release = [&](int order) { tc_commit(&sh->kv_empty[stage_of(order)]); };
        // one key tile: the outputs of tile i, and the scores of tile i + 1 before or after
        auto step = [&](int i) {
            const bool more = i + 1 < tiles;
            if (!two) {
                if (more) {
                    if (!wait_tile(k_order(i + 1))) return false;
                    scores(q0, (i + 1) & 1, i + 1);
                    release(k_order(i + 1));
                    if (i + 2 == tiles) tc_commit(&sh->q_empty[q0]);
                }
                if (!wait_probs(i & 1) || !wait_tile(v_order(i, tiles)) || !outputs(0, i & 1, i)) return false;
            } else {
                if (!wait_probs(0) || !wait_tile(v_order(i, tiles)) || !outputs(0, 0, i)) return false;
                if (more) {
                    if (!wait_tile(k_order(i + 1))) return false;
                    scores(0, 0, i + 1);
                }
                if (!wait_probs(1) || !outputs(1, 1, i)) return false;
                if (more) {
                    scores(1, 1, i + 1);
                    release(k_order(i + 1));
                    if (i + 2 == tiles) {
                        tc_commit(&sh->q_empty[0]);
                        tc_commit(&sh->q_empty[1]);
                    }
                }
            }
            release(v_order(i, tiles));
            return true;
        };
        bool ok = true;
        if (leader) {
            for (int t = 0; t < (two ? 2 : 1) && ok; ++t) {
                const int qb = two ? t : q0;
                ok = lane_wait(sh, &sh->q_full[qb], q_uses[qb]++ & 1);
            }
            ok = ok && wait_tile(k_order(0));
            if (ok) {
                scores(q0, 0, 0);
                if (two) scores(1, 1, 0);
                release(k_order(0));
                if (tiles == 1) {
                    tc_commit(&sh->q_empty[q0]);
                    if (two) tc_commit(&sh->q_empty[1]);
                }
            }
            for (int i = 0; i < tiles && ok; ++i) ok = step(i);
        }
        __syncwarp();
        if (__any_sync(0xFFFFFFFFu, !ok)) break;
        before += 2 * tiles;
        if (!two) next ^= 1;
    }
    // no product outlives the CTA, whichever way the loop ended
    if (leader) {
        tc_commit(&sh->drain);
        wait_drained(&sh->drain, 0);
    }
    __syncwarp();
}

// A vector's stored outputs, with the non-finite values that mend_tiles took out of
// the rows first .. last of the arrays.  Called for items that hold such values alone.
__device__ __noinline__ void add_nonfinite(const AttnPromptArgs &a, int j, int first, int last, uint16_t *out) {
    for (int d = 0; d < kHeadDim; ++d) {
        float x = 0.f;
        for (int t = first; t <= last; ++t) {
            const uint16_t v = a.v[(size_t)t * a.ldv + j * kHeadDim + d];
            if ((v & 0x7F80u) == 0x7F80u) x += __uint_as_float(uint32_t(v) << 16);
        }
        if (x != 0.f) out[d] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(uint32_t(out[d]) << 16) + x));
    }
}

__device__ void softmax(const KernelArgs &k, Shared *sh, uint32_t tmem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wg = warp >> 2;
    const uint32_t my_lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t t_o = tmem + kTmemO + wg * kHeadDim + my_lanes;
    const int v = 32 * (warp & 3) + lane, my_row = v / k.a.group, my_head = v - my_row * k.a.group;
    unsigned s_uses[2] = {0, 0}, o_uses = 0;     // the second group counts its barrier in s_uses[1]
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (!warp_wait(sh, &sh->item_full[slot], (n / kRing) & 1)) return;
        const Item &it = sh->item[slot];        // read where it is needed: registers are short
        if (it.n_rows == 0) return;
        auto release = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
        };
        const bool two = it.n_rows > k.rows_tile;
        const int tiles = (it.i0 + it.n_rows + kTile - 1) / kTile;
        if (wg == 1 && !two) {
            release();
            continue;
        }
        const int n_here = min(k.rows_tile, it.n_rows - wg * k.rows_tile);      // rows of this tile
        const bool active = 32 * (warp & 3) < n_here * k.a.group;
        const int lim = it.i0 + wg * k.rows_tile + min(my_row, n_here - 1);     // the last row this vector sees
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < tiles; ++i) {
            const int buf = two ? wg : i & 1;
            if (!warp_wait(sh, &sh->s_full[wg ? 2 : buf], s_uses[buf]++ & 1)) return;
            bool seen = i == 0;     // whether the previous tile's product into the output is known to be done
            if (active) {
                tc_fence_after();
                const uint32_t t_s = tmem + kTmemS + buf * kTile + my_lanes;
                const int last = lim - i * kTile;
                uint32_t x[64], y[64];
                tc_ld32(t_s, x);
                tc_ld32(t_s + 32, x + 32);
                tc_ld32(t_s + 64, y);
                tc_ld32(t_s + 96, y + 32);
                tc_wait_ld();
                tc_pin32(x);
                tc_pin32(x + 32);
                tc_pin32(y);
                tc_pin32(y + 32);
                if (__any_sync(0xFFFFFFFFu, last < kTile - 1)) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        x[c] = c <= last ? x[c] : 0xFF800000u;
                        y[c] = 64 + c <= last ? y[c] : 0xFF800000u;
                    }
                }
                float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    mt[(c >> 1) & 1] = max3(mt[(c >> 1) & 1], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
                    mt[2 + ((c >> 1) & 1)] = max3(mt[2 + ((c >> 1) & 1)], __uint_as_float(y[c]), __uint_as_float(y[c + 1]));
                }
                const float top = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
                const bool moved = top > m + kMaxSlack;     // true for the first visible scores (m = -inf)
                float scale = 1.f;
                if (moved) {
                    scale = ex2_approx((m - top) * kScaleLog2);
                    m = top;
                    l *= scale;
                }
                if (i > 0 && __any_sync(0xFFFFFFFFu, moved)) {
                    // outputs so far, once the last product into them is done
                    if (!warp_wait(sh, &sh->o_done[wg], (o_uses + i - 1) & 1)) return;
                    seen = true;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tc_ld32(t_o + 32 * c, o);
                        tc_wait_ld();
                        tc_pin32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
                        tc_st32(t_o + 32 * c, o);
                    }
                    tc_wait_st();
                }
                const float mc = m == -INFINITY ? 0.f : m * kScaleLog2;
                const uint64_t scale2 = pack2(kScaleLog2, kScaleLog2), shift2 = pack2(-mc, -mc);
                uint64_t sum2[2] = {0ull, 0ull};
                auto weigh = [&](uint32_t *s, int h) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        float a, b;
                        unpack2(fma2(pack2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, shift2), a, b);
                        a = ex2_approx(a);
                        b = ex2_approx(b);
                        sum2[c & 1] = add2(sum2[c & 1], pack2(a, b));
                        // weights meet V as bf16 (off by at most 2^-8 of each, half a step);
                        // the sum keeps them whole
                        const __nv_bfloat162 pk = __floats2bfloat162_rn(a, b);
                        s[c] = *reinterpret_cast<const uint32_t *>(&pk);
                    }
                    tc_st32(t_s + 32 * h, s);
                };
                weigh(x, 0);
                tc_wait_st();       // the product with the first 64 keys may start
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full[buf][0]);
                weigh(y, 1);
                float s0, s1, s2, s3;
                unpack2(sum2[0], s0, s1);
                unpack2(sum2[1], s2, s3);
                l += (s0 + s1) + (s2 + s3);
                tc_wait_st();
            } else if (lane == 0) {
                mbar_arrive(&sh->p_full[buf][0]);
            }
            // every phase is waited on; this one was over long ago
            if (!seen && !warp_wait(sh, &sh->o_done[wg], (o_uses + i - 1) & 1)) return;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->p_full[buf][1]);
        }
        o_uses += tiles;
        if (!warp_wait(sh, &sh->o_done[wg], (o_uses - 1) & 1)) return;
        if (!active) {
            release();
            continue;
        }
        tc_fence_after();
        const bool store = my_row < n_here;
        const bool bad = *reinterpret_cast<volatile int *>(&sh->bad[slot]) != 0;
        const float inv = __frcp_rn(l);
        const size_t row = (size_t)(it.seq0 + it.i0 + wg * k.rows_tile + my_row);
        uint4 *dst = reinterpret_cast<uint4 *>(k.a.out + row * k.a.ldo + (size_t)(it.j * k.a.group + my_head) * kHeadDim);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tc_ld32(t_o + 32 * c, o);
            tc_wait_ld();
            tc_pin32(o);
            if (store) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w[4];
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[8 * e + 2 * f]) * inv,
                                                                      __uint_as_float(o[8 * e + 2 * f + 1]) * inv);
                        w[f] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    dst[4 * c + e] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
        tc_fence_before();      // the reads of O precede this warp's next arrival on p_full
        if (bad && store) add_nonfinite(k.a, it.j, it.seq0 + it.i0 + 1, it.seq0 + lim, reinterpret_cast<uint16_t *>(dst));
        release();
    }
}

__global__ void __launch_bounds__(kCtaThreads, 1) attn_prompt_kernel(const __grid_constant__ KernelArgs k) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_tiles = smem, *stages = smem + 2 * kTileBytes;
    Shared *sh = reinterpret_cast<Shared *>(stages + size_t(kStages) * kTileBytes);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh->kv_full[i], 1);
            mbar_init(&sh->kv_empty[i], 1);
        }
        for (int i = 0; i < kMends; ++i) mbar_init(&sh->mend_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->q_full[i], 1);
            mbar_init(&sh->q_empty[i], 1);
            mbar_init(&sh->p_full[i][0], 4);
            mbar_init(&sh->p_full[i][1], 4);
            mbar_init(&sh->o_done[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh->item_full[i], 1);
            mbar_init(&sh->item_empty[i], kReaders);
        }
        for (int i = 0; i < 3; ++i) mbar_init(&sh->s_full[i], 1);
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tc_alloc(&sh->tmem, kTmemCols);
    if (warp == kProducerWarp && (threadIdx.x & 31) < 3) prefetch_tensormap(&k.q + (threadIdx.x & 31));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    grid_dependency_wait();     // the rows and starts come from the preceding grids
    grid_launch_dependents();
    if (warp < kSoftmaxWarps) {
        regs_raise<kRegsSoftmax>();
        softmax(k, sh, tmem);
    } else {
        regs_lower<kRegsOther>();
        if (warp == kProducerWarp)
            produce(k, sh, q_tiles, stages);
        else if (warp == kMmaWarp)
            multiply(k, sh, q_tiles, stages, tmem);
        else
            mend_tiles(sh, stages);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) {
        if (sh->abort) set_error(k.a.err, kDevTimeout);
        if (atomicAdd(k.next + 1, 1u) == gridDim.x - 1) {       // every CTA has taken its last item
            k.next[0] = 0u;
            k.next[1] = 0u;
        }
    }
    if (warp == kMmaWarp) tc_dealloc(tmem, kTmemCols);
}

// Innermost first: a head's 128 elements, heads, rows.
bool encode_rows(CUtensorMap *m, const uint16_t *base, int heads, int rows, int ld, int box_heads, int box_rows,
                 const char **why) {
    return encode_tiles(m, base, {cuuint64_t(kHeadDim), cuuint64_t(heads), cuuint64_t(rows)},
                        {cuuint64_t(kHeadDim) * 2, cuuint64_t(ld) * 2}, {64, cuuint32_t(box_heads), cuuint32_t(box_rows)},
                        CU_TENSOR_MAP_SWIZZLE_128B, why);
}

}  // namespace

// The item counters lie in the status block, where no operator has scratch.
constexpr size_t kCountersAt = 192;

cudaError_t launch_attn_prompt(const AttnPromptArgs &a, cudaStream_t s, const char **why) {
    static std::atomic<bool> opted_in[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !opted_in[dev]) {
        e = cudaFuncSetAttribute(attn_prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemBytes));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) opted_in[dev] = true;
    }
    KernelArgs k{};
    k.a = a;
    k.rows_tile = kTile / a.group;
    k.next = reinterpret_cast<unsigned *>(static_cast<char *>(a.ws) + kCountersAt);
    const int sms = device_sm_count();
    auto items = [&](int rows_item) {       // at most: where the sequences lie is on the device
        return (long long)a.n_kv * ((a.rows + rows_item - 1) / rows_item + a.n_seq);
    };
    // two tiles share each K and V tile, but one tile an item where two would leave SMs without any
    k.rows_item = items(2 * k.rows_tile) >= sms ? 2 * k.rows_tile : k.rows_tile;
    if (!encode_rows(&k.q, a.q, a.n_kv * a.group, a.rows, a.ldq, a.group, k.rows_tile, why) ||
        !encode_rows(&k.k, a.k, a.n_kv, a.rows, a.ldk, 1, kTile, why) ||
        !encode_rows(&k.v, a.v, a.n_kv, a.rows, a.ldv, 1, kTile, why))
        return cudaErrorInvalidValue;
    const long long most = items(k.rows_item);
    return launch_pdl(attn_prompt_kernel, dim3(unsigned(most < sms ? most : sms)), dim3(kCtaThreads), kSmemBytes, s, k);
}

}  // namespace tfk
