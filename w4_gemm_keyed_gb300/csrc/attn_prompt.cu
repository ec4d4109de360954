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
// The flow through a CTA: attn_flow.cuh.
//
// What bounds it (GB300, call after call on the same inputs): long prompts, the tensor cores
// and the power limit (32768 rows x 32 heads 5,250 us, 1.68 PFLOP/s; the softmax and its hand-overs make a step of two tiles and 80
// keys 1,640 cycles where its products take 1,440); pages, the change from item to item, 2,000 to 3,000 cycles (2047 rows x 64
// heads 56 us, five of up to 4099 rows x 20 heads 230); many short ones, one thread's finding and copying of an item, 5,000 to 8,000
// cycles, next to 40 us of HBM time (48 of up to 301 rows x 64 heads 63 us); one token, the launch (5.6 us).
#include <atomic>

#include "attn_prompt.cuh"
#include "attn_flow.cuh"
#include "w4_gemm.cuh"

namespace tfk {

namespace {

using namespace flow;

constexpr int kStages = 3;              // K tiles, and V tiles, in shared memory
constexpr int kQueries = 3;             // query tiles in shared memory
static_assert(kQueries == kStages, "one ring length");
constexpr int kProducerWarp = 8, kScoreWarp = 9, kMendWarp = 11;
constexpr int kStoreWarp = 12, kStoreWarps = 4;
constexpr int kCtaThreads = 512;
constexpr int kRegsSoftmax = 168, kRegsOther = 88;
static_assert(256 * kRegsSoftmax + (kCtaThreads - 256) * kRegsOther <= kCtaThreads * 128, "register split");
constexpr int kReaders = kSoftmaxWarps + 2 + kStoreWarps;       // of the item ring

struct Item : ItemBase {
    int j;              // KV head
    int i0;             // first row's place in its sequence
    int seq0;           // the sequence's first row in the arrays
};

struct KernelArgs {
    CUtensorMap q, k, v;
    AttnPromptArgs a;
    int rows_tile;      // rows per tile of 128 vectors
    int rows_item;      // rows per item: one or two tiles
    unsigned *next;     // items taken beyond the first of each CTA, and CTAs done; both zero between calls
};

// ------------------------------------------------------------------ item order
// Items in descending order of their place in their sequences (so of their cost):
// level by level, at each level the sequences that reach it, heads fastest.  The set
// of sequences that reach a level changes only where one of them ends, so a whole run of levels is
// found with one pass over the sequences.  A warp's work, in step.
struct Sequences {      // in shared memory
    int start[kMaxSeqs + 1], levels[kMaxSeqs];      // first rows; items a head
};

struct __align__(16) Shared : SharedBase<Item, kStages, kStages, kQueries> {
    // Of a tile's latest two items: the sums of the next item may follow before these are
    // looked at, but not those of the one after.
    uint64_t l_full[2][2];
    float l[2][2][kTile];
    Sequences sequences;
};
constexpr size_t kSmemBytes = size_t(kQueries) * kTileBytes + size_t(2 * kStages) * kKeyBytes + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct Finder {
    const KernelArgs &k;
    Sequences &all;
    int next_level, high, count;
    unsigned first, end;

    // Whole warp.  Starts that fall or lie outside the rows: no items.
    __device__ Finder(const KernelArgs &args, Sequences &place) : k(args), all(place), next_level(-1), high(0), count(0), first(0), end(0) {
        const int lane = threadIdx.x & 31;
        bool bad = false;
        int top = 0;
#pragma unroll 1
        for (int s = lane; s < k.a.n_seq; s += 32) {
            const long long x = k.a.starts[s], y = k.a.starts[s + 1];
            if (x < 0 || y < x || y > k.a.rows) {
                bad = true;
                continue;
            }
            all.start[s] = int(x);
            if (s + 1 == k.a.n_seq) all.start[s + 1] = int(y);
            all.levels[s] = int(idx_div(unsigned(y - x) + k.rows_item - 1, k.rows_item));
            top = max(top, all.levels[s]);
        }
        __syncwarp();
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
#pragma unroll 1
            for (int s = lane; s < k.a.n_seq; s += 32) {
                const int n = all.levels[s];
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
        const unsigned per_level = unsigned(count) * unsigned(k.a.n_kv), down = idx_div(i - first, per_level);
        const unsigned rest = i - first - down * per_level;
        int nth = int(idx_div(rest, k.a.n_kv));
        it.j = int(rest) - nth * k.a.n_kv;
        it.i0 = (high - int(down)) * k.rows_item;
#pragma unroll 1
        for (int s0 = 0;; s0 += 32) {       // the nth sequence that reaches the level
            unsigned reach = __ballot_sync(0xFFFFFFFFu, s0 + lane < k.a.n_seq && all.levels[min(s0 + lane, kMaxSeqs - 1)] > high);
            const int here = __popc(reach);
            if (nth >= here) {
                nth -= here;
                continue;
            }
            const bool me = (reach >> lane & 1u) && __popc(reach & ((1u << lane) - 1u)) == nth;
            const int s = s0 + __ffs(__ballot_sync(0xFFFFFFFFu, me)) - 1;
            it.seq0 = all.start[s];
            it.n_rows = min(k.rows_item, all.start[s + 1] - it.seq0 - it.i0);
            it.n_keys = it.i0 + it.n_rows;
            return it;
        }
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

__device__ void produce(const KernelArgs &k, Shared *sh, uint8_t *q_tiles, uint8_t *stages) {
    const int lane = threadIdx.x & 31, g = k.a.group;
    Finder finder(k, sh->sequences);
    unsigned i = blockIdx.x;
    unsigned queries = 0, keys = 0, values = 0;     // tiles so far
    unsigned mended = 0;            // of them V tiles to mend
    unsigned to_mend = 0;           // bit st: the last tile of V stage st is one
    bool ok = true;
    // One thread.  The stage of a ring's next tile, once it is free.
    auto room = [&](uint64_t *empty, unsigned n) {
        const int st = n % kStages;
        ok = ok && (n < unsigned(kStages) || lane_idle_wait(sh, &empty[st], (n / kStages - 1) & 1));
        return st;
    };
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        const Item it = finder.find(i);
        if (n >= kRing && !warp_idle_wait(sh, &sh->item_empty[slot], (n / kRing - 1) & 1)) break;
        unsigned taken = 0;
        if (lane == 0) {
            sh->item[slot] = it;
            sh->bad[slot] = 0;
            mbar_arrive(&sh->item_full[slot]);
            if (it.n_rows) taken = atomicAdd(k.next, 1u);       // the item after this one
        }
        if (it.n_rows == 0) break;
        if (lane == 0) {
            const int n_keys = it.n_keys, tiles = (n_keys + kKeys - 1) / kKeys;
#pragma unroll 1
            for (int t = 0; t < 2 && t * k.rows_tile < it.n_rows; ++t) {
                const int buf = room(sh->q_empty, queries);
                if (!ok) break;
                ++queries;
                const int row = it.seq0 + it.i0 + t * k.rows_tile;
                load_queries(q_tiles + buf * kTileBytes, &k.q, it.j * g, row, k.rows_tile * g, &sh->q_full[buf]);
            }
            auto load = [&](const CUtensorMap *map, uint8_t *dst, int key, uint64_t *bar) {
                mbar_arrive_expect_tx(bar, kKeyBytes);
                tma_load_4d(dst, map, 0, it.seq0 + key, it.j, 0, bar);
            };
#pragma unroll 1
            for (int t = 0; t <= tiles && ok; ++t) {        // K(0), then K(t) and V(t - 1)
                if (t < tiles) {
                    const int st = room(sh->k_empty, keys);
                    if (!ok) break;
                    ++keys;
                    load(&k.k, stages + size_t(st) * kKeyBytes, t * kKeys, &sh->k_full[st]);
                }
                if (t > 0) {
                    const int st = room(sh->v_empty, values), key = (t - 1) * kKeys;
                    if (!ok) break;
                    ++values;
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
    auto drain = [&](uint64_t *full, unsigned n, unsigned stages_of, unsigned except) {
#pragma unroll 1
        for (unsigned t = n > stages_of ? n - stages_of : 0; t < n; ++t)
            if (!(except >> (t % stages_of) & 1u)) wait_drained(&full[t % stages_of], (t / stages_of) & 1);
    };
    drain(sh->k_full, keys, kStages, 0u);
    drain(sh->v_full, values, kStages, to_mend);
    drain(sh->mend_full, mended, kMends, 0u);
    drain(sh->q_full, queries, kQueries, 0u);
    sh->mend[mended % kMends].stage = -1;
    mbar_arrive(&sh->mend_full[mended % kMends]);
}

// Stored outputs, with the sums of the non-finite values that their vectors see in their place.  Whole warp:
// all its vectors see the rows first .. common of the arrays, this lane's those up to `last`.  Few registers: it runs
// in the storing warps' share of them (43 by itself; 59 with eight loads at once).
__device__ __noinline__ void put_seen_nonfinite(const AttnPromptArgs &a, int j, int first, int common, int last, bool mine,
                                                uint16_t *out) {
    const int lane = threadIdx.x & 31;
    constexpr int kAtOnce = 4;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const uint16_t *const v = a.v + (size_t)j * kHeadDim;
#pragma unroll 1
    for (int row0 = first + (lane >> 4); row0 <= common; row0 += 2 * kAtOnce) {
        uint4 w[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)       // the last row again changes nothing
            w[i] = *reinterpret_cast<const uint4 *>(v + (size_t)min(row0 + 2 * i, common) * a.ldv + 8 * (lane & 15));
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) add_nonfinite(w[i], x);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] += __shfl_xor_sync(0xFFFFFFFFu, x[e], 16);
#pragma unroll 1
    for (int c = 0; c < kHeadDim / 8; ++c) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xFFFFFFFFu, x[e], c);
        if (!mine) continue;
        for (int t = common + 1; t <= last; ++t)
            add_nonfinite(*reinterpret_cast<const uint4 *>(v + (size_t)t * a.ldv + 8 * c), y);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (y[e] != 0.f) out[8 * c + e] = __bfloat16_as_ushort(__float2bfloat16_rn(y[e]));
    }
}

// Outputs over their weight sums, as bf16: a thread per vector, 32 bytes (a whole
// sector) at a time.  Looking whether one of them is not finite takes 0.2 us of a call's 5.6, and 0 to 1 % of
// longer ones (12000 rows x 16 heads 1.5 %); a test of each word's bits took as long.  With every value of v infinite, 32768 rows x 32
// heads take 33 ms (5.2).
__device__ void store_outputs(const KernelArgs &k, Shared *sh, uint32_t tmem) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) - kStoreWarp, v = 32 * quarter + lane;
    const int g = k.a.group, my_row = v / g;
    const size_t place = (size_t)my_row * k.a.ldo + (size_t)(v - my_row * g) * kHeadDim;
    const bool sectors = ((reinterpret_cast<uintptr_t>(k.a.out) | size_t(k.a.ldo) * 2) & 31) == 0;
    unsigned uses0 = 0, uses1 = 0;
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (!warp_idle_wait(sh, &sh->item_full[slot], (n / kRing) & 1)) return;
        const Item it = sh->item[slot];
        if (it.n_rows == 0) return;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            const int n_here = min(k.rows_tile, it.n_rows - t * k.rows_tile);
            if (n_here <= 0) continue;
            const unsigned use = t ? uses1++ : uses0++;
            if (!warp_idle_wait(sh, &sh->l_full[use & 1][t], (use >> 1) & 1) || !warp_idle_wait(sh, &sh->o_last[t], use & 1)) return;
            if (32 * quarter < n_here * g) {
                tc_fence_after();
                const uint32_t t_o = tmem + kTmemO + t * kHeadDim + (uint32_t(32 * quarter) << 16);
                const float l = sh->l[use & 1][t][v], inv = __frcp_rn(l);
                uint32_t probe = 0u;
                const int row0 = it.seq0 + it.i0 + t * k.rows_tile;
                uint16_t *const out = k.a.out + (size_t)row0 * k.a.ldo + (size_t)it.j * g * kHeadDim + place;
#pragma unroll 1
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
                        probe = probe_finite(w[e], probe);
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
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->o_free[t]);
                // the next products need not wait for what follows; `l` has been read, and the slot is kept
                const bool mine = my_row < n_here;
                if (__any_sync(0xFFFFFFFFu, mine && l > 0.f && (bf16x2_nonfinite(probe) ||
                                                               *reinterpret_cast<volatile int *>(&sh->bad[slot]) != 0)))
                    put_seen_nonfinite(k.a, it.j, it.seq0, row0 + 32 * quarter / g, row0 + my_row, mine && l > 0.f, out);
            } else if (lane == 0) {
                mbar_arrive(&sh->o_free[t]);
            }
            __syncwarp();
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
        sh->init(1, kReaders, kStoreWarps);
        for (int i = 0; i < 4; ++i) mbar_init(&sh->l_full[i >> 1][i & 1], 4);
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
        unsigned items = 0;     // of this warp's tile
        const auto sight = [&](int, const Item &it, int tile, int n_here, int mine, int first, int last) {
            const int row0 = it.i0 + tile * k.rows_tile;        // row i of the sequence sees keys 0 .. i
            return Sight{row0 + min(mine, n_here - 1), row0 + min(first, n_here - 1), row0 + min(last, n_here - 1)};
        };
        // No one reads the sums of the tile's item before the last any more: the products of
        // the last one, seen done by now, had waited for that.
        softmax<false>(sh, k.rows_tile, k.a.group, tmem, sight, [&](int, int tile, int, float, float l, unsigned) {
            sh->l[items & 1][tile][threadIdx.x & 127] = l;
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(&sh->l_full[items & 1][tile]);
            ++items;
            return true;
        });
    } else {
        regs_lower<kRegsOther>();
        if (warp >= kStoreWarp)
            store_outputs(k, sh, tmem);
        else if (warp == kProducerWarp)
            produce(k, sh, q_tiles, stages);
        else if (warp == kMendWarp)
            mend_tiles(sh, stages + size_t(kStages) * kKeyBytes);
        else if (elect_one()) {
            if (warp == kScoreWarp)
                issue_scores(sh, k.rows_tile, q_tiles, stages, tmem);
            else
                issue_outputs(sh, k.rows_tile, stages + size_t(kStages) * kKeyBytes, tmem);
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

// Innermost first: half a head's elements, rows, heads, halves: a tile's two halves in one copy.
bool encode_keys(CUtensorMap *m, const uint16_t *base, int heads, int rows, int ld, const char **why) {
    return encode_tiles<4>(m, base, {64, cuuint64_t(rows), cuuint64_t(heads), 2},
                           {cuuint64_t(ld) * 2, cuuint64_t(kHeadDim) * 2, 128}, {64, kKeys, 1, 2}, CU_TENSOR_MAP_SWIZZLE_128B, why);
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
    if (!encode_queries(&k.q, a.q, a.n_kv * a.group, a.rows, a.ldq, a.group, k.rows_tile, why) ||
        !encode_keys(&k.k, a.k, a.n_kv, a.rows, a.ldk, why) ||
        !encode_keys(&k.v, a.v, a.n_kv, a.rows, a.ldv, why))
        return cudaErrorInvalidValue;
    const long long most = items(k.rows_item);
    return launch_pdl(attn_prompt_kernel, dim3(unsigned(most < sms ? most : sms)), dim3(kCtaThreads), kSmemBytes, s, k);
}

}  // namespace tfk
