// Causal attention of whole prompts, packed one after the other.
//
// Row i of a sequence attends over its rows 0 .. i:
//   s_t = q . k_t / sqrt(128),  o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m).
//
// A tile is 128 query vectors: whole rows of one KV head's query heads (a vector is a
// row and a head), so that a K and V tile in shared memory serves every head that reads it
// and short prompts fill their tiles.  An item is two neighbouring tiles (one where
// there are few); each vector folds the keys of its sequence in ascending order,
// kKeys at a time from the sequence's first row, with a running maximum, and no other vector's
// values ever mix with its own: its bits depend on its own query and keys alone.
// Scores and outputs run on tcgen05: S = Q K^T with both operands in shared memory
// and S in tensor memory, then P (bf16) times V with P read from tensor memory.
// Persistent CTAs take items from a counter, the longest first over all sequences.
//
// Keys are taken 80 at a time because tensor memory (512 columns) then holds, next to two tiles'
// outputs (256), their scores (160) and their weights (80) apart: the next scores are
// computed while this step's weights are formed, and the products never wait for the
// chain scores - softmax - weights of one step.
#include <atomic>

#include <cuda_bf16.h>

#include "attn_prompt.cuh"
#include "attn_tiles.cuh"
#include "w4_gemm.cuh"

namespace tfk {

namespace {

constexpr int kKeys = 80;               // keys of a K or V tile
constexpr int kKeyHalf = kKeys * 128;   // 64 elements of a tile's rows
constexpr int kKeyBytes = 2 * kKeyHalf;
constexpr int kStages = 3;              // K tiles, and V tiles, in shared memory
constexpr int kQueries = 3;             // query tiles in shared memory
constexpr int kRing = 4;                // items known ahead
constexpr int kMends = 4;               // V tiles to mend on their way: at most kStages, and an end mark
constexpr int kSoftmaxWarps = 8, kProducerWarp = 8, kScoreWarp = 9, kOutputWarp = 10, kMendWarp = 11;
constexpr int kStoreWarp = 12, kStoreWarps = 4;
constexpr int kCtaThreads = 512;
constexpr int kRegsSoftmax = 168, kRegsOther = 88;
static_assert(256 * kRegsSoftmax + (kCtaThreads - 256) * kRegsOther <= kCtaThreads * 128, "register split");
constexpr int kReaders = kSoftmaxWarps + 2 + kStoreWarps;       // of the item ring
constexpr uint32_t kTmemCols = 512, kTmemO = 0, kTmemS = 256, kTmemP = kTmemS + 2 * kKeys;
constexpr uint32_t kPStride = (kKeys / 2 + 15) / 16 * 16;      // columns of a tile's weights
static_assert(kTmemP + 2 * kPStride <= kTmemCols, "tensor memory");
static_assert(kKeyHalf % 1024 == 0 && kKeys % 16 == 0, "whole swizzle atoms and product steps");

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
// barrier waits on every one of its phases, and before the next can end.  Index: tile of an item.
struct __align__(16) Shared {
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], mend_full[kMends];
    uint64_t q_full[kQueries], q_empty[kQueries];
    uint64_t s_full[2], s_free[2], p_full[2], o_done[2];
    // A tile's last product of an item, its sums, its output taken.  The sums of the next
    // item may follow before these are looked at, but not those of the one after.
    uint64_t o_last[2], l_full[2][2], o_free[2];
    uint64_t item_full[kRing], item_empty[kRing], drain[2];
    Item item[kRing];
    Mend mend[kMends];
    int bad[kRing];     // whether a value that only some vectors see is not finite
    float l[2][2][kTile];       // weight sums: of a tile's latest two items
    uint32_t tmem;
    int abort;
};
constexpr size_t kSmemBytes = size_t(kQueries) * kTileBytes + size_t(2 * kStages) * kKeyBytes + sizeof(Shared);
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
    static constexpr int kHeld = 2;         // sequences a lane keeps in registers: the first 64 in all
    const KernelArgs &k;
    int held[kHeld], start[kHeld], rows[kHeld];     // their items a head, first rows and lengths
    int next_level, high, count;
    unsigned first, end;

    __device__ int levels(int n) const { return int(idx_div(unsigned(n) + k.rows_item - 1, k.rows_item)); }    // of n rows
    // f(items a head, first row, length) of this lane's sequences, 32 in step, until f says true
    template <typename F>
    __device__ void each(F f) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (f(held[h], start[h], rows[h])) return;
        for (int s0 = 32 * kHeld; s0 < k.a.n_seq; s0 += 32) {
            const int s = s0 + lane;
            const int x = s < k.a.n_seq ? int(k.a.starts[s]) : 0, n = s < k.a.n_seq ? int(k.a.starts[s + 1]) - x : 0;
            if (f(levels(n), x, n)) return;
        }
    }
    // Whole warp.  Starts that fall or lie outside the rows: no items.
    __device__ explicit Finder(const KernelArgs &args) : k(args), held{}, start{}, rows{}, next_level(-1), high(0), count(0), first(0), end(0) {
        const int lane = threadIdx.x & 31;
        bool bad = false;
        for (int s = lane; s < k.a.n_seq; s += 32) {
            const long long x = k.a.starts[s], y = k.a.starts[s + 1];
            bad |= x < 0 || y < x || y > k.a.rows;
        }
        if (__any_sync(0xFFFFFFFFu, bad)) {
            if (blockIdx.x == 0 && lane == 0) set_error(k.a.err, kDevBadPosition);
            return;
        }
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (lane + 32 * h < k.a.n_seq) {
                start[h] = int(k.a.starts[lane + 32 * h]);
                rows[h] = int(k.a.starts[lane + 32 * h + 1]) - start[h];
                held[h] = levels(rows[h]);
            }
        int top = 0;
        each([&](int n, int, int) {
            top = max(top, n);
            return false;
        });
        next_level = __reduce_max_sync(0xFFFFFFFFu, top) - 1;
    }
    // Whole warp; i never falls from call to call.
    __device__ Item find(unsigned i) {
        const int lane = threadIdx.x & 31;
        Item it{};
        while (i >= end) {
            if (next_level < 0) return it;
            int more = 0, below = 0;
            each([&](int n, int, int) {
                if (n > next_level)
                    ++more;
                else
                    below = max(below, n);
                return false;
            });
            count = __reduce_add_sync(0xFFFFFFFFu, more);
            below = __reduce_max_sync(0xFFFFFFFFu, below);
            first = end;
            end += unsigned(next_level - below + 1) * unsigned(count) * unsigned(k.a.n_kv);
            high = next_level;
            next_level = below - 1;
        }
        const unsigned per_level = unsigned(count) * unsigned(k.a.n_kv), down = idx_div(i - first, per_level);
        const unsigned rest = i - first - down * per_level;
        int nth = int(idx_div(rest, k.a.n_kv));
        it.j = int(rest) - nth * k.a.n_kv;
        it.i0 = (high - int(down)) * k.rows_item;
        each([&](int n, int x, int len) {       // the nth sequence that reaches the level
            const unsigned reach = __ballot_sync(0xFFFFFFFFu, n > high);
            const int here = __popc(reach);
            if (nth < here) {
                const bool me = n > high && __popc(reach & ((1u << lane) - 1u)) == nth;
                const int from = __ffs(__ballot_sync(0xFFFFFFFFu, me)) - 1;
                it.seq0 = __shfl_sync(0xFFFFFFFFu, x, from);
                it.n_rows = min(k.rows_item, __shfl_sync(0xFFFFFFFFu, len, from) - it.i0);
                return true;
            }
            nth -= here;
            return false;
        });
        return it;
    }
};

// ------------------------------------------------------------------ roles
//   warp 8      finds the items and streams their query vectors and K and V tiles by TMA
//   warp 9      issues the products S = Q K^T
//   warp 10     issues the products O += P V
//   warp 11     mends V tiles that reach past what all the item's vectors see
//   warps 0-7   softmax: a thread per vector, four warps a tile of the item (items of one
//               tile leave the other four idle)
//   warps 12-15 scale and store the outputs while the others are at the next item

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

__device__ void produce(const KernelArgs &k, Shared *sh, uint8_t *q_tiles, uint8_t *stages) {
    const int lane = threadIdx.x & 31, g = k.a.group;
    Finder finder(k);
    unsigned i = blockIdx.x;
    unsigned loaded_k = 0, loaded_v = 0, queries = 0;   // tiles so far
    unsigned mended = 0;            // of them V tiles to mend
    unsigned to_mend = 0;           // bit st: the last tile of V stage st is one
    bool ok = true;
    // One thread.  The stage of a ring's next tile, once it is free.
    auto room = [&](uint64_t *empty, unsigned n, int stages_of) {
        const int st = n % stages_of;
        ok = ok && (n < unsigned(stages_of) || lane_wait(sh, &empty[st], (n / stages_of - 1) & 1));
        return st;
    };
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        const Item it = finder.find(i);
        if (n >= kRing && !warp_wait(sh, &sh->item_empty[slot], (n / kRing - 1) & 1)) break;
        unsigned taken = 0;
        if (lane == 0) {
            sh->item[slot] = it;
            sh->bad[slot] = 0;
            mbar_arrive(&sh->item_full[slot]);
            if (it.n_rows) taken = atomicAdd(k.next, 1u);       // the item after this one
        }
        if (it.n_rows == 0) break;
        if (lane == 0) {
            const int n_keys = it.i0 + it.n_rows, tiles = (n_keys + kKeys - 1) / kKeys;
            // A tile of queries is whole rows of the KV head's query heads, one box of (64
            // elements, heads, rows) per half.  Rows of the box past the item's
            // fill vectors that nothing reads: rows of a product never mix.
            for (int t = 0; t < 2 && t * k.rows_tile < it.n_rows; ++t) {
                const int buf = room(sh->q_empty, queries, kQueries);
                if (!ok) break;
                ++queries;
                const int row = it.seq0 + it.i0 + t * k.rows_tile;
                mbar_arrive_expect_tx(&sh->q_full[buf], 2 * uint32_t(k.rows_tile * g) * 128u);
                tma_load_3d(q_tiles + buf * kTileBytes, &k.q, 0, it.j * g, row, &sh->q_full[buf]);
                tma_load_3d(q_tiles + buf * kTileBytes + kHalfBytes, &k.q, 64, it.j * g, row, &sh->q_full[buf]);
            }
            auto load = [&](const CUtensorMap *map, uint8_t *dst, int key, uint64_t *bar) {
                mbar_arrive_expect_tx(bar, kKeyBytes);
                tma_load_3d(dst, map, 0, it.j, it.seq0 + key, bar);
                tma_load_3d(dst + kKeyHalf, map, 64, it.j, it.seq0 + key, bar);
            };
            for (int t = 0; t <= tiles && ok; ++t) {        // K(0), then K(t) and V(t - 1)
                if (t < tiles) {
                    const int st = room(sh->k_empty, loaded_k, kStages);
                    if (!ok) break;
                    ++loaded_k;
                    load(&k.k, stages + size_t(st) * kKeyBytes, t * kKeys, &sh->k_full[st]);
                }
                if (t > 0) {
                    const int st = room(sh->v_empty, loaded_v, kStages), key = (t - 1) * kKeys;
                    if (!ok) break;
                    ++loaded_v;
                    uint64_t *bar = &sh->v_full[st];
                    const int first = max(0, it.i0 + 1 - key);
                    to_mend &= ~(1u << st);
                    if (first < kKeys) {        // past the first row's last key: handed over by the mender
                        const int m = mended++ % kMends;
                        sh->mend[m] = {st, slot, first, min(kKeys, n_keys - key)};
                        to_mend |= 1u << st;
                        bar = &sh->mend_full[m];
                    }
                    load(&k.v, stages + size_t(kStages + st) * kKeyBytes, key, bar);
                }
            }
        }
        __syncwarp();
        if (!__shfl_sync(0xFFFFFFFFu, int(ok), 0)) break;
        i = gridDim.x + __shfl_sync(0xFFFFFFFFu, taken, 0);
    }
    if (lane != 0) return;
    // no copy outlives the CTA
    auto drain = [&](uint64_t *full, unsigned n, int stages_of, unsigned except) {
        for (unsigned t = n > unsigned(stages_of) ? n - stages_of : 0; t < n; ++t)
            if (!(except >> (t % stages_of) & 1u)) wait_drained(&full[t % stages_of], (t / stages_of) & 1);
    };
    drain(sh->k_full, loaded_k, kStages, 0u);
    drain(sh->v_full, loaded_v, kStages, to_mend);
    drain(sh->mend_full, mended, kMends, 0u);
    drain(sh->q_full, queries, kQueries, 0u);
    sh->mend[mended % kMends].stage = -1;
    mbar_arrive(&sh->mend_full[mended % kMends]);
}

// V tiles that hold rows some vectors of the item do not see: rows past the item's
// last become zeros (up to the 16-row step the product reads; they are another sequence's,
// or nobody's), and non-finite elements of rows that only some vectors see become zero, since
// 0 * inf would reach the others; the vectors that see them get them back when
// the output is stored.
__device__ void mend_tiles(Shared *sh, uint8_t *stages) {
    const int lane = threadIdx.x & 31, c = lane & 15;
    constexpr int kAtOnce = 8;          // pairs of rows
    for (unsigned n = 0;; ++n) {
        const int slot = n % kMends;
        if (!warp_wait(sh, &sh->mend_full[slot], (n / kMends) & 1)) return;
        const Mend m = sh->mend[slot];
        if (m.stage < 0) return;
        uint8_t *v = stages + size_t(kStages + m.stage) * kKeyBytes + (c >> 3) * kKeyHalf;
        auto at = [&](int row) { return reinterpret_cast<uint4 *>(v + row * 128 + (((c & 7) ^ (row & 7)) << 4)); };
        const int end = (m.valid + 15) & ~15;
        bool bad = false;
        for (int row0 = m.first + (lane >> 4); row0 < m.valid; row0 += 2 * kAtOnce) {
            uint4 x[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                x[i] = row0 + 2 * i < m.valid ? *at(row0 + 2 * i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (bf16x2_nonfinite(x[i].x) || bf16x2_nonfinite(x[i].y) || bf16x2_nonfinite(x[i].z) || bf16x2_nonfinite(x[i].w)) {
                    *at(row0 + 2 * i) = make_uint4(bf16x2_finite(x[i].x), bf16x2_finite(x[i].y), bf16x2_finite(x[i].z),
                                                   bf16x2_finite(x[i].w));
                    bad = true;
                }
            }
        }
        for (int row = m.valid + (lane >> 4); row < end; row += 2) *at(row) = make_uint4(0u, 0u, 0u, 0u);
        if (bad) *reinterpret_cast<volatile int *>(&sh->bad[m.slot]) = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->v_full[m.stage]);
    }
}

// The items in order, for a role of one thread; what it needs of one.
struct Items {
    const KernelArgs &k;
    Shared *sh;
    Ring<kRing> ring;
    int tiles = 0, n_keys = 0;
    bool two = false;
    __device__ bool next() {        // false: no more, or gave up
        if (!lane_wait(sh, &sh->item_full[ring.at], ring.parity)) return false;
        const Item it = sh->item[ring.at];
        mbar_arrive(&sh->item_empty[ring.at]);
        ring.step();
        two = it.n_rows > k.rows_tile;
        n_keys = it.i0 + it.n_rows;
        tiles = (n_keys + kKeys - 1) / kKeys;
        return it.n_rows != 0;
    }
    __device__ int steps16(int i) const { return (min(kKeys, n_keys - i * kKeys) + 15) >> 4; }
};

// Scores and outputs are issued by two threads, each of which waits for what its own
// products need: every wait and commit costs the thread that issues them some 100 cycles,
// and one thread for both took 2,600 cycles a step of two tiles where the products take 1,450.

// S[t] = Q[t] K(i)^T for the item's one or two tiles t, key tile by key tile (rounded up to 16 keys).
__device__ void issue_scores(const KernelArgs &k, Shared *sh, uint8_t *q_tiles, uint8_t *stages, uint32_t tmem) {
    Items items{k, sh};
    Ring<kStages> tile;
    Ring<kQueries> query;
    uint32_t free_parity[2] = {1u, 1u};     // of a fresh barrier, the phase before the first counts as over
    const uint32_t q_addr = smem_u32(q_tiles), k_addr = smem_u32(stages);
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
__device__ void issue_outputs(const KernelArgs &k, Shared *sh, uint8_t *stages, uint32_t tmem) {
    Items items{k, sh};
    Ring<kStages> tile;
    uint32_t p_parity[2] = {0u, 0u}, free_parity[2] = {1u, 1u};
    const uint32_t v_addr = smem_u32(stages) + kStages * kKeyBytes;
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

__device__ void softmax(const KernelArgs &k, Shared *sh, uint32_t tmem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wg = warp >> 2;
    const uint32_t my_lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t t_o = tmem + kTmemO + wg * kHeadDim + my_lanes, t_s = tmem + kTmemS + wg * kKeys + my_lanes,
                   t_p = tmem + kTmemP + wg * kPStride + my_lanes;
    const int v0 = 32 * (warp & 3), row_first = v0 / k.a.group, row_last = (v0 + 31) / k.a.group,
              my_row = (v0 + lane) / k.a.group;
    const uint64_t scale2 = pack2(kScaleLog2, kScaleLog2);
    unsigned steps = 0, items = 0;  // of this group
    auto hand = [&](uint64_t *bar) {        // what the warp has read or written in tensor memory
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (!warp_wait(sh, &sh->item_full[slot], (n / kRing) & 1)) return;
        const int n_rows = sh->item[slot].n_rows, i0 = sh->item[slot].i0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
        if (n_rows == 0) return;
        const int n_here = min(k.rows_tile, n_rows - wg * k.rows_tile);     // rows of this tile
        if (n_here <= 0) continue;
        const int n_keys = i0 + n_rows, tiles = (n_keys + kKeys - 1) / kKeys;
        const bool active = row_first < n_here;
        // the last row each vector sees: this one, and the warp's least and greatest
        const int row0 = i0 + wg * k.rows_tile, lim = row0 + min(my_row, n_here - 1),
                  lim_first = row0 + min(row_first, n_here - 1), lim_last = row0 + min(row_last, n_here - 1);
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
            } else if (lim_first >= (i + 1) * kKeys - 1) {       // every vector sees every key
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
                const int seen = lim_last < key ? 0 : min(steps16, ((lim_last - key) >> 4) + 1);
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
            // no one reads the sums of the tile's item before the last any more: the products of
            // the last one, seen done above, had waited for that
            if (i + 1 == tiles) {
                sh->l[items & 1][wg][v0 + lane] = l;
                hand(&sh->l_full[items & 1][wg]);
            }
            hand(&sh->p_full[wg]);
        }
        ++items;
    }
}

// Outputs over their weight sums, as bf16: a thread per vector, 32 bytes (a whole
// sector) at a time.
__device__ void store_outputs(const KernelArgs &k, Shared *sh, uint32_t tmem) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) - kStoreWarp, v = 32 * quarter + lane;
    const int g = k.a.group, my_row = v / g;
    const size_t place = (size_t)my_row * k.a.ldo + (size_t)(v - my_row * g) * kHeadDim;
    const bool sectors = ((reinterpret_cast<uintptr_t>(k.a.out) | size_t(k.a.ldo) * 2) & 31) == 0;
    unsigned uses[2] = {0, 0};
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (!warp_wait(sh, &sh->item_full[slot], (n / kRing) & 1)) return;
        const Item it = sh->item[slot];
        if (it.n_rows == 0) return;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int n_here = min(k.rows_tile, it.n_rows - t * k.rows_tile);
            if (n_here <= 0) continue;
            const unsigned use = uses[t]++;
            if (!warp_wait(sh, &sh->l_full[use & 1][t], (use >> 1) & 1) || !warp_wait(sh, &sh->o_last[t], use & 1)) return;
            if (32 * quarter < n_here * g) {
                tc_fence_after();
                const uint32_t t_o = tmem + kTmemO + t * kHeadDim + (uint32_t(32 * quarter) << 16);
                const float inv = __frcp_rn(sh->l[use & 1][t][v]);
                const int row0 = it.seq0 + it.i0 + t * k.rows_tile;
                uint16_t *const out = k.a.out + (size_t)row0 * k.a.ldo + (size_t)it.j * g * kHeadDim + place;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32], w[16];
                    tc_ld32(t_o + 32 * c, o);
                    tc_wait_ld();
                    tc_pin32(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const __nv_bfloat162 h =
                            __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                        w[e] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    if (my_row < n_here) {
                        if (sectors) {
                            st_global_32(out + 32 * c, w);
                            st_global_32(out + 32 * c + 16, w + 8);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<uint4 *>(out + 32 * c + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
                        }
                    }
                }
                tc_fence_before();
                if (*reinterpret_cast<volatile int *>(&sh->bad[slot]) != 0 && my_row < n_here)
                    add_nonfinite(k.a, it.j, it.seq0 + it.i0 + 1, row0 + my_row, out);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->o_free[t]);
        }
        if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
    }
}

__global__ void __launch_bounds__(kCtaThreads, 1) attn_prompt_kernel(const __grid_constant__ KernelArgs k) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_tiles = smem, *stages = smem + kQueries * kTileBytes;
    Shared *sh = reinterpret_cast<Shared *>(stages + size_t(2 * kStages) * kKeyBytes);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh->k_full[i], 1);
            mbar_init(&sh->k_empty[i], 1);
            mbar_init(&sh->v_full[i], 1);
            mbar_init(&sh->v_empty[i], 1);
        }
        for (int i = 0; i < kMends; ++i) mbar_init(&sh->mend_full[i], 1);
        for (int i = 0; i < kQueries; ++i) {
            mbar_init(&sh->q_full[i], 1);
            mbar_init(&sh->q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->s_free[i], 4);
            mbar_init(&sh->p_full[i], 4);
            mbar_init(&sh->o_done[i], 1);
            mbar_init(&sh->o_last[i], 1);
            mbar_init(&sh->l_full[0][i], 4);
            mbar_init(&sh->l_full[1][i], 4);
            mbar_init(&sh->o_free[i], kStoreWarps);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh->item_full[i], 1);
            mbar_init(&sh->item_empty[i], kReaders);
        }
        mbar_init(&sh->drain[0], 1);
        mbar_init(&sh->drain[1], 1);
        sh->abort = 0;
        fence_mbar_init();
    }
    if (warp == kScoreWarp) tc_alloc(&sh->tmem, kTmemCols);
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
        if (warp >= kStoreWarp)
            store_outputs(k, sh, tmem);
        else if (warp == kProducerWarp)
            produce(k, sh, q_tiles, stages);
        else if (warp == kMendWarp)
            mend_tiles(sh, stages);
        else if (elect_one()) {
            if (warp == kScoreWarp)
                issue_scores(k, sh, q_tiles, stages, tmem);
            else
                issue_outputs(k, sh, stages, tmem);
        }
        __syncwarp();
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
    if (warp == kScoreWarp) tc_dealloc(tmem, kTmemCols);
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
        !encode_rows(&k.k, a.k, a.n_kv, a.rows, a.ldk, 1, kKeys, why) ||
        !encode_rows(&k.v, a.v, a.n_kv, a.rows, a.ldv, 1, kKeys, why))
        return cudaErrorInvalidValue;
    const long long most = items(k.rows_item);
    return launch_pdl(attn_prompt_kernel, dim3(unsigned(most < sms ? most : sms)), dim3(kCtaThreads), kSmemBytes, s, k);
}

}  // namespace tfk
