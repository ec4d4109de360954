// Attention of trees of drafted tokens over a shared prefix, their sequences' own entries
// and their paths.
//
// Node i of sequence b (depth d, position pos[b] + d) attends over the prefix's entries
// 0 .. P - 1, its sequence's own entries 0 .. pos[b] - 1 and those of its path's nodes:
//   s_t = q . k_t / sqrt(128),  o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m).
//
// A node's bits must not tell whether an ancestor is a node of this pass or was
// committed before.  So the entries at its last kMaxPath own positions, every node of its path among
// them, are "near": they are one matrix product's keys, in path order.  The others, all of them
// before the root, are "far" and lie on a fixed grid of parts:
// kOwnPart own entries, or of the prefix a length that P and the number of KV heads
// fix.  A far part is folded by the flow of attn_flow.cuh, each vector for itself, and its result stored (maximum m,
// weight sum l, unnormalised output o, fp32); a second kernel works on the near entries and adds up all parts in ascending
// order, the near ones last.  So bits depend on a node's query, position, P and the entries that it sees.
//
// What bounds it (GB300, call after call on the same inputs): many nodes, the tensor cores and what
// storing an item's results takes, 128 KB at 28 bytes a cycle (24 x 64 nodes x 64 heads over 32768 entries 1,075 us: parts 973 at
// 1.50 PFLOP/s, the sum 93 at 5.2 TB/s); few, the steps one SM has in a row (5 x 24 nodes over 8192 41 us: two items of 12
// steps, the sum 11; 3 x 41 nodes x 20 heads over own 12007 31 us) or launches (8 nodes over 300 entries 10.7 us).  E4M3 where nothing is
// expanded first, the chain copy - expand - product - softmax of a step (16 nodes over 30000 50 us, 37 as a bf16 cache).
#include <atomic>

#include "attn_flow.cuh"
#include "attn_tree.cuh"
#include "tree.cuh"
#include "w4_gemm.cuh"

namespace tfk {

namespace {

using namespace flow;

constexpr int kOwnPart = 320;           // own entries per part
// Shared entries per part, at least: an item's results take as long to store as two and a half steps.  With 240: 64 x 64 nodes over
// 500 entries 297 us (225), 32 x 16 over 1000 60 (43), but 8 over 300 9.9 (11.1), 8 over 2000 10.9 (12.7); with 960 30 x 40 over 3000
// 83 (95), 8 over 2000 15.6, 64 x 64 of one head over 1000 23.8 (22.0).
constexpr int kMinPrefixPart = 560;
// Items of a batch that is one pair of tiles, about.  Twice as many: 1 x 16 nodes over 65536 entries 57 us (69), over 30000 8-bit ones
// 37 (51), 4 x 8 over 30000 41 (44), but 24 x 64 over 32768 1,228 (1,074), 16 x 32 over 16461 8-bit ones 297 (257), 8 x 8 over 16000
// 43 (37), 5 x 24 over 8192 48 (41).
constexpr int kPrefixItems = 76;
// An E4M3 prefix is expanded into the workspace first where that pays: it saves every pair of query tiles
// 28 ns per 1,000 entries and head, costs 76 ns and the two further grids 10 us, so from (pairs - 3) x entries x heads = 340,000 on
// (16 x 32 nodes, 16 pairs, over 16461 x 8: 257 us, 297 without; 16 x 8 nodes, 4 pairs, over 16000 x 8: 85, 80 without;
// 32 x 16 nodes, 16 pairs, over 1000 x 8: 55, 51 without).
constexpr long long kExpandWork = 340000;
constexpr int kGroups = 128;            // entries of the table of own items
constexpr int kProducerWarp = 8, kScoreWarp = 9, kMendWarp = 11;
constexpr int kExpandWarp = 12, kExpandWarps = 4;       // E4M3: for K tiles, and as many for V tiles
constexpr int kRawBytes = kKeys * kHeadDim;
static_assert(kOwnPart % kKeys == 0 && kMinPrefixPart % kKeys == 0, "whole key tiles");

// What the cache's format changes: an E4M3 tile (10 KB and 80 scale bytes) is copied into a raw
// stage and expanded into a bf16 tile by four more warps for K, four for V, so the products are those of a
// bf16 cache holding the same values.  Where many items read it, the prefix is expanded into the workspace first.
template <bool E4M3>
struct Form {
    static constexpr int k_stages = 3, v_stages = E4M3 ? 2 : 3;     // bf16 tiles in shared memory
    static constexpr int queries = E4M3 ? 2 : 3;        // query tiles
    static constexpr int raw = E4M3 ? 3 : 0;            // E4M3 K tiles, and V tiles, on their way
    static constexpr int threads = E4M3 ? 640 : 384;
    static constexpr int readers = kSoftmaxWarps + 2 + (E4M3 ? 2 * kExpandWarps : 0);   // of the item ring
    // registers a thread: the softmax warps', the next four's and the expanding ones', together no more than the launch's
    static constexpr int regs_softmax = E4M3 ? 144 : 200, regs_other = E4M3 ? 64 : 104, regs_expand = 64;
    static_assert(256 * regs_softmax + 128 * regs_other + (threads - 384) * regs_expand <= threads * (E4M3 ? 96 : 168), "register split");
};

struct Item : ItemBase {
    int j, b;           // KV head, sequence (-1: prefix)
    int row0, key0;     // first row, first entry
    int lim0;           // last entry of the item that a root sees (own), n_keys - 1 (prefix)
    int block;          // of its results: (slot, KV head)
};

// Results: values [slot][n_kv][32 quads of columns][vectors][4], so that the 32 vectors of a warp store and load
// 512 consecutive bytes (with a vector's 128 values side by side, 32 bytes a thread, an item of 5 x 24 nodes took
// 15 us, 12 of them for its stores), and maxima and sums [slot][n_kv][vectors].  Slots: the prefix's parts, then own ones.
struct Plan {
    int rows, rows_tile;        // of the batch; of a tile of query vectors
    int rows_item, own_rows_item;       // of an item over the prefix, over own entries: one or two tiles
    int pairs, own_pairs;       // items over all rows, and over a sequence's
    int part, n_parts;          // the prefix's parts: length and number
    int own_parts_max;
    int expanded;               // whether an E4M3 prefix is expanded into the workspace first
};

__host__ __device__ inline int prefix_part(int prefix_len, int n_kv) {
    const int parts = kPrefixItems / n_kv > 0 ? kPrefixItems / n_kv : 1, even = (prefix_len - 1) / parts + 1;
    const long long part = ((long long)even + kKeys - 1) / kKeys * kKeys;
    return int(part < kMinPrefixPart ? kMinPrefixPart : (part > 0x7FFFFFFF ? 0x7FFFFFFF / kKeys * kKeys : part));
}

// sms: SMs that items of one and of two tiles are weighed for; no size in the workspace follows it.
Plan plan_of(const KvBatch &own, int prefix_len, int group, int n, int sms) {
    Plan p;
    p.rows = own.n_seq * n;
    p.rows_tile = kTile / group;
    p.part = prefix_len > 0 ? prefix_part(prefix_len, own.n_kv) : kMinPrefixPart;
    p.n_parts = prefix_len > 0 ? (prefix_len - 1) / p.part + 1 : 0;
    p.own_parts_max = (own.max_len + kOwnPart - 1) / kOwnPart;
    // Two tiles share each K and V tile, and a step of both takes 1.7 times as long as of one alone: one tile an
    // item where the SMs are then done sooner (4 x 8 nodes over 30000 entries, 72 items of two: 40-44 us, 54 as two; 8 x 8 over 16000,
    // 144: 37 as two, 47 as one).  Own parts: at most as many as the caches hold.
    auto items = [](int rows, int rows_item) { return (rows + rows_item - 1) / rows_item; };
    const int both = 2 * p.rows_tile;
    auto rows_item = [&](long long parts, int rows) {
        auto rounds = [&](int of) { return (parts * items(rows, of) + sms - 1) / sms; };
        return 17 * rounds(both) <= 10 * rounds(p.rows_tile) ? both : p.rows_tile;
    };
    p.rows_item = rows_item((long long)p.n_parts * own.n_kv, p.rows);
    p.own_rows_item = rows_item((long long)p.own_parts_max * own.n_kv * own.n_seq, n);
    p.pairs = items(p.rows, p.rows_item);
    p.own_pairs = items(n, p.own_rows_item);
    p.expanded = own.format == kKvE4m3 && (long long)(items(p.rows, both) - 3) * prefix_len * own.n_kv >= kExpandWork;
    return p;
}

// Entries of a head of the expanded prefix, and its bytes (K and V).
inline int expanded_len(int prefix_len) { return (prefix_len + 7) & ~7; }
size_t expanded_bytes(const Plan &p, int prefix_len, int n_kv) {
    return p.expanded ? size_t(4) * expanded_len(prefix_len) * n_kv * kHeadDim : 0;
}

long long slots_of(const Plan &p, int n_kv, int group) {
    return (long long)(p.n_parts + p.own_parts_max) * n_kv * p.rows * group;
}

struct KernelArgs {
    CUtensorMap map[5];     // prefix K, V; own K, V (bf16 caches); queries
    AttnTreeArgs a;
    Plan p;
    float *values;          // [slots][128]
    float2 *ml;             // [slots]: (maximum score, weight sum)
    unsigned *next;         // items taken beyond the first of each CTA; zero between calls
    int prefix_parts;       // that this kernel works on: all or none
    bool own_parts;         // whether it works on them
    bool overlaps;          // whether the preceding grid works on the other parts: nothing of its is read
};

template <bool E4M3>
struct __align__(16) Shared : SharedBase<Item, Form<E4M3>::k_stages, Form<E4M3>::v_stages, Form<E4M3>::queries> {
    uint64_t raw_full[2][3], raw_empty[2][3];   // K, V
    unsigned before[kGroups + 1];       // own items of the sequence groups before each
    int8_t depth[kRing][kMaxNodes];     // of an own item's nodes
};
// query tiles, bf16 stages, raw stages, their scales, then Shared
template <bool E4M3>
constexpr size_t kSmemBytes = size_t(Form<E4M3>::queries) * kTileBytes + size_t(Form<E4M3>::k_stages + Form<E4M3>::v_stages) * kKeyBytes +
                              size_t(2 * Form<E4M3>::raw) * (kRawBytes + kTile) + sizeof(Shared<E4M3>);
static_assert(kSmemBytes<false> <= 227 * 1024 && kSmemBytes<true> <= 227 * 1024, "shared memory");

// Two parts' factors in their sum, and its maximum.
struct Factors {
    float top, a, b;
};
__device__ __forceinline__ Factors factors(float ma, float mb) {
    const float top = fmaxf(ma, mb), t = top == -INFINITY ? 0.f : top;
    return {top, ex2_approx((ma - t) * kScaleLog2), ex2_approx((mb - t) * kScaleLog2)};
}
__device__ __forceinline__ float fold(const Factors &f, float x, float y) { return fmaf(y, f.b, __fmul_rn(x, f.a)); }

__device__ __forceinline__ float4 fold(const Factors &f, const float4 &x, const float4 &y) {
    return make_float4(fold(f, x.x, y.x), fold(f, x.y, y.y), fold(f, x.z, y.z), fold(f, x.w, y.w));
}

// ------------------------------------------------------------------ item order
// The prefix's parts first (the longest), pairs of tiles fastest so that the CTAs
// working on one part read it from L2; then own parts, heads fastest.
__device__ int own_items(const KernelArgs &k, int b, bool report) {     // a head's, over the entries before the root
    const long long p = seq_position(k.a.pos, b, k.a.n, k.a.own.max_len, k.a.err, report);
    return p < 0 ? 0 : int((p + kOwnPart - 1) / kOwnPart) * k.p.own_pairs;
}

__device__ Item item_of(const KernelArgs &k, const unsigned *before, unsigned i, int group_seqs) {
    Item it{};
    const unsigned n_kv = k.a.own.n_kv, pairs = k.p.pairs;
    const unsigned n_prefix = k.prefix_parts * n_kv * pairs;
    if (i < n_prefix) {
        it.block = idx_div(i, pairs);
        const int c = idx_div(it.block, n_kv);
        it.j = it.block - c * n_kv;
        it.b = -1;
        it.row0 = (i - it.block * pairs) * k.p.rows_item;
        it.n_rows = min(k.p.rows_item, k.p.rows - it.row0);
        it.key0 = c * k.p.part;
        it.n_keys = min(k.p.part, k.a.prefix_len - it.key0);
        it.lim0 = it.n_keys - 1;
        return it;
    }
    i -= n_prefix;
    const int n_groups = (k.a.own.n_seq + group_seqs - 1) / group_seqs;
    if (i >= before[n_groups] * n_kv) return it;
    int u = idx_div(i, n_kv);
    it.j = i - u * n_kv;
    int lo = 0, hi = n_groups - 1;      // last group whose items start at or before u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= unsigned(u))
            lo = mid;
        else
            hi = mid - 1;
    }
    u -= before[lo];
    int b = lo * group_seqs;
    for (int n; u >= (n = own_items(k, b, false)); ++b) u -= n;
    const long long p = k.a.pos[b];
    const int c = idx_div(u, k.p.own_pairs), first = (u - c * k.p.own_pairs) * k.p.own_rows_item;
    it.block = (k.p.n_parts + c) * n_kv + it.j;
    it.b = b;
    it.row0 = b * k.a.n + first;
    it.n_rows = min(k.p.own_rows_item, k.a.n - first);
    it.key0 = c * kOwnPart;
    it.n_keys = int(min((long long)kOwnPart, p - it.key0));
    it.lim0 = int(p - kMaxPath - it.key0);
    return it;
}

// ------------------------------------------------------------------ roles, beside those of the flow
//   warp 8        finds the items and streams their query vectors and K and V tiles by TMA
//   warps 0-7     also store an item's results
//   warps 12-19   (E4M3) expand K tiles (12-15) and V tiles
template <bool E4M3>
__device__ void produce(const KernelArgs &k, Shared<E4M3> *sh, uint8_t *q_tiles, uint8_t *stages, uint8_t *raw) {
    using F = Form<E4M3>;
    const int lane = threadIdx.x & 31, n_seq = k.a.own.n_seq, g = k.a.group;
    const int group_seqs = (n_seq + kGroups - 1) / kGroups;
    const int n_groups = (n_seq + group_seqs - 1) / group_seqs;
    int total = 0;
    for (int g0 = 0; g0 < n_groups; g0 += 32) {
        int n = 0;
        for (int b = (g0 + lane) * group_seqs; k.own_parts && b < min(n_seq, (g0 + lane + 1) * group_seqs); ++b)
            n += own_items(k, b, blockIdx.x == 0);
        int sum = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += t;
        }
        if (g0 + lane < n_groups) sh->before[g0 + lane] = total + sum - n;
        total += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) sh->before[n_groups] = total;
    __syncwarp();

    unsigned i = blockIdx.x;
    unsigned loaded_k = 0, loaded_v = 0, queries = 0;   // tiles so far
    unsigned mended = 0;            // of them V tiles to mend
    unsigned to_mend = 0;           // bit st: the last tile of V stage st is one
    constexpr int kRaw = E4M3 ? F::raw : 1;
    bool ok = true;
    // One thread.  The stage of a ring's next tile, once it is free.
    auto room = [&](uint64_t *empty, unsigned n, int stages_of) {
        const int st = n % stages_of;
        ok = ok && (n < unsigned(stages_of) || lane_idle_wait(sh, &empty[st], (n / stages_of - 1) & 1));
        return st;
    };
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        const Item it = item_of(k, sh->before, i, group_seqs);
        if (n >= kRing && !warp_idle_wait(sh, &sh->item_empty[slot], (n / kRing - 1) & 1)) break;
        if (it.n_rows && it.b >= 0) {
            int d[2];       // of no tree: anything small; what its rows get is not used
            tree_depths(k.a.parents + (size_t)it.b * k.a.n, k.a.n, d);
            sh->depth[slot][lane] = int8_t(d[0]);
            sh->depth[slot][lane + 32] = int8_t(d[1]);
            __syncwarp();
        }
        unsigned taken = 0;
        if (lane == 0) {
            sh->item[slot] = it;
            sh->bad[slot] = 0;
            mbar_arrive(&sh->item_full[slot]);
            if (it.n_rows) taken = atomicAdd(k.next, 1u);       // the item after this one
        }
        if (it.n_rows == 0) break;
        if (lane == 0) {
            const bool own = it.b >= 0;
            const int tiles = (it.n_keys + kKeys - 1) / kKeys, outer = own ? it.b * k.a.own.n_kv + it.j : it.j;
#pragma unroll 1
            for (int t = 0; t < 2 && t * k.p.rows_tile < it.n_rows; ++t) {
                const int buf = room(sh->q_empty, queries, F::queries);
                if (!ok) break;
                ++queries;
                const int row = it.row0 + t * k.p.rows_tile;
                load_queries(q_tiles + buf * kTileBytes, &k.map[4], it.j * g, row, k.p.rows_tile * g, &sh->q_full[buf]);
            }
            // one tile of entries key0 + key ..
            auto load = [&](bool is_v, int key) {
                const int row = it.key0 + key;
                if constexpr (E4M3) {
                    unsigned &loaded = is_v ? loaded_v : loaded_k;
                    const int st = room(sh->raw_empty[is_v], loaded, kRaw), at = (is_v ? kRaw : 0) + st;
                    if (!ok) return;
                    ++loaded;
                    const KvBatch &cache = own ? k.a.own : k.a.prefix;
                    const uint32_t rows = uint32_t(min(kKeys, it.n_keys - key)), scales = (rows + 15u) & ~15u;
                    const size_t entry = (size_t)outer * cache.max_len + (size_t)row;
                    uint64_t *bar = &sh->raw_full[is_v][st];
                    mbar_arrive_expect_tx(bar, rows * kHeadDim + scales);
                    bulk_g2s(raw + size_t(at) * kRawBytes,
                             static_cast<const uint8_t *>(is_v ? cache.v : cache.k) + entry * kHeadDim, rows * kHeadDim, bar);
                    bulk_g2s(raw + size_t(2 * kRaw) * kRawBytes + at * kTile, (is_v ? cache.v_scale : cache.k_scale) + entry,
                             scales, bar);
                } else {
                    unsigned &loaded = is_v ? loaded_v : loaded_k;
                    const int st = room(is_v ? sh->v_empty : sh->k_empty, loaded, is_v ? F::v_stages : F::k_stages);
                    if (!ok) return;
                    ++loaded;
                    uint64_t *bar = is_v ? &sh->v_full[st] : &sh->k_full[st];
                    uint8_t *dst = stages + size_t(is_v ? F::k_stages + st : st) * kKeyBytes;
                    if (is_v) {
                        to_mend &= ~(1u << st);
                        const int first = max(0, it.lim0 + 1 - key);
                        if (own && first < kKeys) {     // past the last entry that every node sees: handed over by the mender
                            const int m = mended++ % kMends;
                            sh->mend[m] = {st, slot, first, min(kKeys, it.n_keys - key)};
                            to_mend |= 1u << st;
                            bar = &sh->mend_full[m];
                        }
                    }
                    const CUtensorMap *map = &k.map[(own ? 2 : 0) + (is_v ? 1 : 0)];
                    mbar_arrive_expect_tx(bar, kKeyBytes);
                    tma_load_4d(dst, map, 0, row, outer, 0, bar);
                }
            };
#pragma unroll 1
            for (int t = 0; t <= tiles && ok; ++t) {        // K(0), then K(t) and V(t - 1)
                if (t < tiles) load(false, t * kKeys);
                if (t > 0 && ok) load(true, (t - 1) * kKeys);
            }
        }
        __syncwarp();
        if (!__shfl_sync(0xFFFFFFFFu, int(ok), 0)) break;
        i = gridDim.x + __shfl_sync(0xFFFFFFFFu, taken, 0);
    }
    if (lane != 0) return;
    // no copy outlives the CTA
    auto drain = [&](uint64_t *full, unsigned count, int stages_of, unsigned except) {
        for (unsigned t = count > unsigned(stages_of) ? count - stages_of : 0; t < count; ++t)
            if (!(except >> (t % stages_of) & 1u)) wait_drained(&full[t % stages_of], (t / stages_of) & 1);
    };
    if constexpr (E4M3) {
        drain(sh->raw_full[0], loaded_k, kRaw, 0u);
        drain(sh->raw_full[1], loaded_v, kRaw, 0u);
    } else {
        drain(sh->k_full, loaded_k, F::k_stages, 0u);
        drain(sh->v_full, loaded_v, F::v_stages, to_mend);
        drain(sh->mend_full, mended, kMends, 0u);
        sh->mend[mended % kMends].stage = -1;
        mbar_arrive(&sh->mend_full[mended % kMends]);
    }
    drain(sh->q_full, queries, F::queries, 0u);
}

// E4M3 tiles -> bf16 tiles, eight lanes an entry.  Rows of a V tile past the
// part's last entry become zeros up to the 16-row step the product reads, and so
// do entries marked NaN that some nodes do not see (0 * NaN would reach those;
// the nodes that see them get the NaN back when the result is stored).
__device__ void expand_tiles(Shared<true> *sh, const bool is_v, uint8_t *tiles_out, const uint8_t *raw) {
    using F = Form<true>;
    constexpr int kRows = 4 * kExpandWarps, kSteps = kKeys / kRows;    // rows the warps take at a time
    static_assert(kRows % 8 == 0 && kKeys % kRows == 0, "a thread's rows share their place in the swizzle");
    const int lane = threadIdx.x & 31, tid = threadIdx.x & (32 * kExpandWarps - 1), group = tid & 7, row0 = tid >> 3;
    const uint8_t *scales = raw + size_t(2 * F::raw) * kRawBytes + (is_v ? F::raw * kTile : 0);
    raw += is_v ? F::raw * kRawBytes : 0;
    uint64_t *const raw_full = sh->raw_full[is_v], *const raw_empty = sh->raw_empty[is_v];
    uint64_t *const full = is_v ? sh->v_full : sh->k_full, *const empty = is_v ? sh->v_empty : sh->k_empty;
    Ring<F::raw> from;
    const int stages = is_v ? F::v_stages : F::k_stages;
    int at = 0;
    uint32_t parity = 1u;   // of a fresh barrier, the phase before the first counts as over
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (!warp_wait(sh, &sh->item_full[slot], (n / kRing) & 1)) return;
        const int n_rows = sh->item[slot].n_rows, n_keys = sh->item[slot].n_keys, lim0 = sh->item[slot].lim0;
        if (n_rows == 0) return;
        const int tiles = (n_keys + kKeys - 1) / kKeys;
        for (int t = 0; t < tiles; ++t) {
            const int key = t * kKeys, valid = min(kKeys, n_keys - key);
            const int fill = is_v ? (valid + 15) & ~15 : valid, hidden = lim0 + 1 - key;
            if (!warp_wait(sh, &raw_full[from.at], from.parity)) return;
            if (!warp_wait(sh, &empty[at], parity)) return;
            const uint8_t *src = raw + size_t(from.at) * kRawBytes + row0 * kHeadDim + 16 * group;
            const uint8_t *sc = scales + from.at * kTile + row0;
            uint8_t *dst = tiles_out + size_t(at) * kKeyBytes + row0 * 128 + ((group ^ (row0 & 7)) << 4);
            const bool whole = valid == kKeys && !(is_v && hidden < kKeys);     // nothing to leave out
            uint4 w[kSteps];
            uint32_t f[kSteps];
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                w[i] = *reinterpret_cast<const uint4 *>(src + i * kRows * kHeadDim);
                f[i] = sc[i * kRows];
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int row = row0 + i * kRows;
                if (!whole) {
                    if (row >= fill) break;
                    if (row >= valid || (is_v && f[i] == uint32_t(kScaleNan) && row >= hidden)) {
                        if (row < valid) *reinterpret_cast<volatile int *>(&sh->bad[slot]) = 1;
                        w[i] = make_uint4(0u, 0u, 0u, 0u);
                        f[i] = 0u;
                    }
                }
                const uint32_t factor = e4m3_factor(f[i]);
                uint4 lo, hi;
                e4m3_expand(w[i].x, factor, lo.x, lo.y);
                e4m3_expand(w[i].y, factor, lo.z, lo.w);
                e4m3_expand(w[i].z, factor, hi.x, hi.y);
                e4m3_expand(w[i].w, factor, hi.z, hi.w);
                *reinterpret_cast<uint4 *>(dst + i * kRows * 128) = lo;
                *reinterpret_cast<uint4 *>(dst + i * kRows * 128 + kKeyHalf) = hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[at]);
                mbar_arrive(&raw_empty[from.at]);
            }
            from.step();
            if (++at == stages) {
                at = 0;
                parity ^= 1u;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
    }
}

// Nodes that see an own entry with non-finite values get them back: they had been left out of the
// product.  The kernel that adds up the parts then finds such an output (put_seen_nonfinite).  out: a
// stored result, its quads `step` apart; first .. last: the item's entries in question.
template <bool E4M3>
__device__ __noinline__ void add_nonfinite(const AttnTreeArgs &a, int b, int j, int key0, int first, int last, float4 *out,
                                           size_t step) {
    const size_t base = (size_t)(b * a.own.n_kv + j) * a.own.max_len + (size_t)key0;
    for (int d = 0; d < kHeadDim; ++d) {
        float x = 0.f;
        for (int t = first; t <= last; ++t) {
            const size_t entry = base + t;
            if constexpr (E4M3) {
                if (a.own.v_scale[entry] == kScaleNan) x = __uint_as_float(0x7FC00000u);
            } else {
                const uint16_t v =
                    static_cast<const uint16_t *>(a.own.v)[entry * kHeadDim + 8 * ((d >> 3) ^ int(entry & 7)) + (d & 7)];
                if ((v & 0x7F80u) == 0x7F80u) x += __uint_as_float(uint32_t(v) << 16);
            }
        }
        if (x != 0.f) reinterpret_cast<float *>(out + (d >> 2) * step)[d & 3] += x;
    }
}

// The last entry of the item that a row's node sees.
template <typename SHARED>
__device__ __forceinline__ int last_seen(const SHARED *sh, const KernelArgs &k, int slot, const Item &it, int row) {
    return it.b < 0 ? it.lim0 : it.lim0 + sh->depth[slot][it.row0 + row - it.b * k.a.n];
}

// An item's results, by the warps of its softmax: a thread per vector.
template <bool E4M3>
__device__ bool store_results(const KernelArgs &k, Shared<E4M3> *sh, uint32_t tmem, int slot, int t, int n_here, float m,
                              float l, unsigned steps) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, v = 32 * quarter + lane;
    const int g = k.a.group, my_row = v / g, n_vec = k.p.rows * g;
    if (!warp_wait(sh, &sh->o_done[t], (steps - 1) & 1)) return false;
    if (32 * quarter < n_here * g) {
        tc_fence_after();
        const uint32_t t_o = tmem + kTmemO + t * kHeadDim + (uint32_t(32 * quarter) << 16);
        const Item &it = sh->item[slot];
        const bool mine = my_row < n_here;
        const size_t block = it.block;
        const int at = (it.row0 + t * k.p.rows_tile) * g + v;
        float4 *const out = reinterpret_cast<float4 *>(k.values) + block * 32 * n_vec + at;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tc_ld32(t_o + 32 * c, o);
            tc_wait_ld();
            tc_pin32(o);
            if (c == 3) {       // the next item's products may begin
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->o_free[t]);
            }
            if (mine) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    out[(size_t)(8 * c + e) * n_vec] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            }
        }
        if (mine) {
            k.ml[block * n_vec + at] = make_float2(m, l);
            if (*reinterpret_cast<volatile int *>(&sh->bad[slot]) != 0)
                add_nonfinite<E4M3>(k.a, it.b, it.j, it.key0, max(0, it.lim0 + 1),
                                    min(it.n_keys - 1, last_seen(sh, k, slot, it, t * k.p.rows_tile + my_row)), out, n_vec);
        }
    } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->o_free[t]);
    }
    return true;
}

template <bool E4M3>
__global__ void __launch_bounds__(Form<E4M3>::threads, 1) attn_tree_kernel(const __grid_constant__ KernelArgs k) {
    using F = Form<E4M3>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_tiles = smem, *stages = smem + F::queries * kTileBytes, *raw = stages + size_t(F::k_stages + F::v_stages) * kKeyBytes;
    uint8_t *const v_tiles = stages + size_t(F::k_stages) * kKeyBytes;
    Shared<E4M3> *sh = reinterpret_cast<Shared<E4M3> *>(raw + size_t(2 * F::raw) * (kRawBytes + kTile));
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        sh->init(E4M3 ? kExpandWarps : 1, F::readers, 4);
        for (int i = 0; i < 2 * F::raw; ++i) {
            mbar_init(&sh->raw_full[i & 1][i >> 1], 1);
            mbar_init(&sh->raw_empty[i & 1][i >> 1], kExpandWarps);
        }
        fence_mbar_init();
    }
    if (warp == kScoreWarp) tc_alloc(&sh->tmem, kTmemCols);
    if (warp == kProducerWarp && (threadIdx.x & 31) < 5) {
        const int m = threadIdx.x & 31;
        if (m == 4 || (!E4M3 && (m < 2 ? k.prefix_parts > 0 : k.own_parts))) prefetch_tensormap(&k.map[m]);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    // Queries, positions, parents and entries come from the preceding grids; the other parts' grid had waited
    // for them when it let this one start.
    if (!k.overlaps) grid_dependency_wait();
    grid_launch_dependents();
    if (warp < kSoftmaxWarps) {
        regs_raise<F::regs_softmax>();
        const auto sight = [&](int slot, const Item &it, int tile, int n_here, int mine, int, int) {
            const int last = last_seen(sh, k, slot, it, tile * k.p.rows_tile + min(mine, n_here - 1));
            if (it.b < 0) return Sight{last, last, last};
            return Sight{last, __reduce_min_sync(0xFFFFFFFFu, last), __reduce_max_sync(0xFFFFFFFFu, last)};
        };
        softmax<true>(sh, k.p.rows_tile, k.a.group, tmem, sight, [&](int slot, int tile, int n_here, float m, float l, unsigned steps) {
            return store_results<E4M3>(k, sh, tmem, slot, tile, n_here, m, l, steps);
        });
    } else {
        if (E4M3 && warp >= kExpandWarp) {
            regs_lower<F::regs_expand>();
            if constexpr (E4M3) {
                const bool is_v = warp >= kExpandWarp + kExpandWarps;
                expand_tiles(sh, is_v, is_v ? v_tiles : stages, raw);
            }
        } else {
            regs_lower<F::regs_other>();
        }
        if (E4M3 && warp >= kExpandWarp) {
        } else if (warp == kProducerWarp) {
            produce<E4M3>(k, sh, q_tiles, stages, raw);
        } else if (warp == kMendWarp) {
            if constexpr (!E4M3) mend_tiles(sh, v_tiles);
        } else if (elect_one()) {
            if (warp == kScoreWarp)
                issue_scores(sh, k.p.rows_tile, q_tiles, stages, tmem);
            else
                issue_outputs(sh, k.p.rows_tile, v_tiles, tmem);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && sh->abort) set_error(k.a.err, kDevTimeout);
    if (warp == kScoreWarp) tc_dealloc(tmem, kTmemCols);
    if (k.overlaps) grid_dependency_wait();     // what waits for this grid waits for that one too
}

// ------------------------------------------------------------------ an E4M3 prefix as bf16
// Eight lanes an entry, entries in the layout of a bf16 cache.  HBM bounds it: 129 bytes read and 256 written.
constexpr int kExpandEntries = 128;     // a CTA's

__global__ void __launch_bounds__(256) expand_prefix_kernel(KvBatch c, int len, int out_len, uint4 *k_out, uint4 *v_out) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int group = threadIdx.x & 7, row0 = blockIdx.x * kExpandEntries + (threadIdx.x >> 3), j = blockIdx.y;
    const uint8_t *codes = static_cast<const uint8_t *>(blockIdx.z ? c.v : c.k) + (size_t)j * c.max_len * kHeadDim;
    const uint8_t *scales = (blockIdx.z ? c.v_scale : c.k_scale) + (size_t)j * c.max_len;
    uint4 *out = (blockIdx.z ? v_out : k_out) + (size_t)j * out_len * 16;
    constexpr int kSteps = kExpandEntries / 32;
    uint4 w[kSteps];
    uint32_t f[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int row = min(row0 + 32 * i, len - 1);
        w[i] = *reinterpret_cast<const uint4 *>(codes + (size_t)row * kHeadDim + 16 * group);
        f[i] = scales[row];
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int row = row0 + 32 * i;
        if (row >= len) break;
        const uint32_t factor = e4m3_factor(f[i]);
        uint4 lo, hi;
        e4m3_expand(w[i].x, factor, lo.x, lo.y);
        e4m3_expand(w[i].y, factor, lo.z, lo.w);
        e4m3_expand(w[i].z, factor, hi.x, hi.y);
        e4m3_expand(w[i].w, factor, hi.z, hi.w);
        out[(size_t)row * 16 + (group ^ (row & 7))] = lo;
        out[(size_t)row * 16 + 8 + (group ^ (row & 7))] = hi;
    }
}

// ------------------------------------------------------------------ near entries, and the sum
// A CTA takes up to VECS vectors (whole nodes) of one KV head.  First the near entries, before the
// attention grid has ended: a warp a node, at most 16 keys in path order, one matrix product (bf16 operands, fp32
// sums) for the scores of its heads and one for their outputs.  Then the far results are added up, the near ones last:
// 256 threads, some quads of columns each.  It reads 520 bytes per vector and slot, and nothing else counts where
// there are many.  With few vectors, the loads that follow one another do: SPLIT CTAs then take a part of the columns each (and
// work on the near entries as often), and keep as many times more slots on their way.
constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps;
constexpr int kNearPitch = kHeadDim + 4;        // floats: lanes that read a quad of consecutive vectors meet no bank twice

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool E4M3>
__device__ __forceinline__ uint4 cache_chunk(const void *data, const uint8_t *scale, size_t entry, int c) {   // elements 8c .. 8c + 7
    uint4 x;
    if constexpr (E4M3) {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(data) + entry * kHeadDim + 16 * (c & 7) +
                                                         8 * (c >> 3));
        const uint32_t f = e4m3_factor(scale[entry]);
        e4m3_expand(w.x, f, x.x, x.y);
        e4m3_expand(w.y, f, x.z, x.w);
    } else {
        x = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(data) + entry * kHeadDim + 8 * (c ^ int(entry & 7)));
    }
    return x;
}

template <int VECS>
struct __align__(16) JoinShared {
    float near[VECS][kNearPitch];      // near outputs; then, as bf16, the rows' outputs
    float2 ml[VECS];
    int depth[VECS];                   // of the nodes; -1: idle sequence, no tree or unused row
    uint4 v[VECS < kJoinWarps ? VECS : kJoinWarps][kMaxPath][16];      // a node's near values, chunk c of row t at c XOR (t % 8)
};

// Where a node is in its tree.  Lane i holds nodes i and i + 32.
struct Node {
    int b, node, depth;     // depth -1: idle sequence, no tree or unused row
    long long pos;
    int above[2];           // parents (the root's: itself)
};

// Whole warp.
__device__ __forceinline__ Node find_node(const AttnTreeArgs &a, int row, bool report) {
    const int lane = threadIdx.x & 31;
    Node t;
    t.b = idx_div(row, a.n);
    t.node = row - t.b * a.n;
    t.pos = seq_position(a.pos, t.b, a.n, a.own.max_len, a.err, false);
    const int32_t *parents = a.parents + (size_t)t.b * a.n;
    int d[2];
    const bool tree = tree_depths(parents, a.n, d);
    if (!tree && t.pos >= 0 && t.node == 0 && report && lane == 0) set_error(a.err, kDevBadTree);
    const int lo = __shfl_sync(0xFFFFFFFFu, d[0], t.node & 31), hi = __shfl_sync(0xFFFFFFFFu, d[1], t.node & 31);
    t.depth = tree && t.pos >= 0 ? (t.node < 32 ? lo : hi) : -1;
#pragma unroll
    for (int h = 0; h < 2; ++h) t.above[h] = lane + 32 * h < a.n ? max(0, parents[lane + 32 * h]) : 0;
    return t;
}

// One node's near entries; whole warp.  Rows of the products are the group's heads, a lane's are lane / 4 and that + 8.
template <bool E4M3, int VECS>
__device__ void near_entries(const AttnTreeArgs &a, JoinShared<VECS> *sh, const Node &t, int j, int nth, uint4 (*s_v)[16]) {
    const int lane = threadIdx.x & 31, g = a.group, r = lane >> 2, c4 = lane & 3, b = t.b, row = t.b * a.n + t.node;
    const long long pos = t.pos;
    auto of = [](const int (&v)[2], int i) {
        const int lo = __shfl_sync(0xFFFFFFFFu, v[0], i & 31), hi = __shfl_sync(0xFFFFFFFFu, v[1], i & 31);
        return i < 32 ? lo : hi;
    };
    // lane t < near: the entry at own position first + t, of a node `up` steps above where it is one of the path
    const int near = int(min((long long)kMaxPath, pos + t.depth + 1));
    const long long first = pos + t.depth + 1 - near;
    int up = max(0, near - 1 - lane), at = t.node;
    int above[2] = {t.above[0], t.above[1]};
#pragma unroll
    for (int s = 0; s < 4; ++s) {       // above: 2^s steps
        const int higher = of(above, at);
        if (up >> s & 1) at = higher;
        const int u0 = of(above, above[0]), u1 = of(above, above[1]);
        above[0] = u0;
        above[1] = u1;
    }
    const long long y = first + lane;
    const int my_entry = int(y < pos ? y : pos + at);
    const size_t base = (size_t)(b * a.own.n_kv + j) * a.own.max_len;

    // Queries and keys: a lane's 16-byte chunk 4i + c4 gives four pairs, the operands of two steps of 16 elements; the sums
    // take the elements in another order than memory has them, the same for both.
    uint4 q[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[h][i] = r + 8 * h < g ? *reinterpret_cast<const uint4 *>(a.q + (size_t)row * a.ldq +
                                                                       (size_t)(j * g + r + 8 * h) * kHeadDim + 8 * (4 * i + c4))
                                    : make_uint4(0u, 0u, 0u, 0u);
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int n = 0; n < 2; ++n) {       // keys 8n .. 8n + 7, the lane's is 8n + r
        const size_t e = base + __shfl_sync(0xFFFFFFFFu, my_entry, 8 * n + r);
        uint4 k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            k[i] = 8 * n + r < near ? cache_chunk<E4M3>(a.own.k, a.own.k_scale, e, 4 * i + c4) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mma_bf16(s[n], q[0][i].x, q[1][i].x, q[0][i].y, q[1][i].y, k[i].x, k[i].y);
            mma_bf16(s[n], q[0][i].z, q[1][i].z, q[0][i].w, q[1][i].w, k[i].z, k[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < kMaxPath / 2; ++i) {
        const int key = 2 * i + (lane >> 4), c = lane & 15;
        const size_t e = base + __shfl_sync(0xFFFFFFFFu, my_entry, key);
        s_v[key][c ^ (key & 7)] = key < near ? cache_chunk<E4M3>(a.own.v, a.own.v_scale, e, c) : make_uint4(0u, 0u, 0u, 0u);
    }
    __syncwarp();
    // weights: s[n][2h + i] is head r + 8h and key 8n + 2 c4 + i
    uint32_t w[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (8 * n + 2 * c4 + i >= near) s[n][2 * h + i] = -INFINITY;
                m = fmaxf(m, s[n][2 * h + i]);
            }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const float mc = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float x = ex2_approx((s[n][2 * h] - mc) * kScaleLog2), z = ex2_approx((s[n][2 * h + 1] - mc) * kScaleLog2);
            l += x + z;
            // weights meet V as bf16 (off by at most 2^-8 of each, half a step); the sums keep them whole
            const __nv_bfloat162 pk = __floats2bfloat162_rn(x, z);
            w[n][h] = *reinterpret_cast<const uint32_t *>(&pk);
        }
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
        if (c4 == 0 && r + 8 * h < g) sh->ml[nth * g + r + 8 * h] = make_float2(m, l);
    }
    // outputs, 16 columns at a time
    const int key = lane & 15;
    const uint32_t v_row = smem_u32(&s_v[key][0]);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        uint32_t v[4];      // keys 0-7 and 8-15 of columns 16n .., then of columns 16n + 8 ..
        ldsm_x4_trans(v_row + 16 * ((2 * n + (lane >> 4)) ^ (key & 7)), v);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            mma_bf16(o, w[0][0], w[0][1], w[1][0], w[1][1], v[2 * i], v[2 * i + 1]);
            const int col = 16 * n + 8 * i + 2 * c4;
            if (r < g) *reinterpret_cast<float2 *>(&sh->near[nth * g + r][col]) = make_float2(o[0], o[1]);
            if (r + 8 < g) *reinterpret_cast<float2 *>(&sh->near[nth * g + r + 8][col]) = make_float2(o[2], o[3]);
        }
    }
    __syncwarp();       // the next node's values may come
}

// The sums of the non-finite values that row `row` (a node's) attends over take the place of its outputs of `quads` quads of
// columns; bf16 caches.
__device__ __noinline__ void put_seen_nonfinite(const AttnTreeArgs &a, int j, int row, int quad, int quads, uint16_t *out) {
    const int b = row / a.n;
    const int32_t *parents = a.parents + (size_t)b * a.n;
    const int pos = int(a.pos[b]);      // the node is one of a tree, so the position is a good one
    const uint16_t *const own = static_cast<const uint16_t *>(a.own.v) + (size_t)(b * a.own.n_kv + j) * a.own.max_len * kHeadDim;
#pragma unroll 1
    for (int i = 0; i < quads; ++i) {
        float4 x = cached_nonfinite(own, 0, pos - 1, quad + i);
        if (a.prefix_len > 0)
            x = add4(x, cached_nonfinite(static_cast<const uint16_t *>(a.prefix.v) + (size_t)j * a.prefix.max_len * kHeadDim, 0,
                                         a.prefix_len - 1, quad + i));
        int node = row - b * a.n;
        for (; node > 0; node = parents[node])      // a parent's number is lower
            x = add4(x, cached_nonfinite(own, pos + node, pos + node, quad + i));
        put_nonfinite(out + 4 * i, add4(x, cached_nonfinite(own, pos, pos, quad + i)));
    }
}

template <bool E4M3, int VECS, int SPLIT, int BLOCKS>
__global__ void __launch_bounds__(kJoinThreads, BLOCKS) attn_tree_join_kernel(const __grid_constant__ AttnTreeArgs a, Plan p,
                                                                         const float *results, const float2 *ml,
                                                                         unsigned *next) {
    constexpr int kQuads = VECS / 8 / SPLIT;        // a thread's: `quad` and the ones after it
    extern __shared__ __align__(1024) uint8_t smem[];
    JoinShared<VECS> *sh = reinterpret_cast<JoinShared<VECS> *>(smem);
    const int warp = threadIdx.x >> 5, g = a.group, j = blockIdx.y, n_kv = a.own.n_kv;
    const int mine = threadIdx.x % VECS, quad = (blockIdx.z * (kJoinThreads / VECS) + threadIdx.x / VECS) * kQuads;
    const int nodes = VECS / g, row0 = blockIdx.x * nodes, here = min(nodes, p.rows - row0), n_vec = p.rows * g;
    Node t{};
    for (int i = warp; i < here; i += kJoinWarps) {
        t = find_node(a, row0 + i, j == 0 && blockIdx.z == 0);
        if ((threadIdx.x & 31) == 0) sh->depth[i] = t.depth;
    }
    __syncthreads();
    // warps without a node go on meanwhile
    for (int i = warp; i < here; i += kJoinWarps) {
        if (warp + kJoinWarps < here) t = find_node(a, row0 + i, false);        // not the one just found
        if (t.depth >= 0) near_entries<E4M3>(a, sh, t, j, i, sh->v[warp]);
    }
    // The results come from the attention grid; all else from before it, which it had
    // waited for when it let this grid start.
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x == 0 && j == 0 && blockIdx.z == 0 && threadIdx.x == 0) next[0] = next[1] = 0u;
    const int nth = mine / g, depth = nth < here ? sh->depth[nth] : -1;
    float4 sum[kQuads];
    float l = 1.f;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY;
    if (depth >= 0) {
        const long long far = a.pos[idx_div(row0 + nth, a.n)] + depth + 1 - kMaxPath;       // own entries that lie farther
        const int n = p.n_parts + (far > 0 ? int((far + kOwnPart - 1) / kOwnPart) : 0);
        const int v = row0 * g + mine;
        const float2 *my_ml = ml + (size_t)j * n_vec + v;
        const float4 *x = reinterpret_cast<const float4 *>(results) + ((size_t)j * 32 + quad) * n_vec + v;
        const size_t step = (size_t)n_kv * n_vec;
        l = 0.f;
        auto add = [&](const float2 &part, const float4 (&y)[kQuads]) {
            const Factors f = factors(m, part.x);
            m = f.top;
            l = fold(f, l, part.y);
#pragma unroll
            for (int i = 0; i < kQuads; ++i) sum[i] = fold(f, sum[i], y[i]);
        };
        constexpr int kAhead = (BLOCKS == 2 ? 16 : 8) / kQuads;     // slots on their way
        float2 w[kAhead];
        float4 y[kAhead][kQuads];
        for (int c = 0; c < n; c += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (c + u < n) {
                    w[u] = *my_ml;
#pragma unroll
                    for (int i = 0; i < kQuads; ++i) y[u][i] = __ldcs(x + (size_t)i * n_vec);
                    my_ml += step;
                    x += step * 32;
                }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (c + u < n) add(w[u], y[u]);
        }
    }
    __syncthreads();    // the near entries' results are there
    if (depth >= 0) {
        const Factors f = factors(m, sh->ml[mine].x);
        l = fold(f, l, sh->ml[mine].y);
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            sum[i] = fold(f, sum[i], *reinterpret_cast<const float4 *>(&sh->near[mine][4 * (quad + i)]));
    }
    __syncthreads();    // the near outputs are read
    uint16_t *const rows = reinterpret_cast<uint16_t *>(&sh->near[0][0]);
    constexpr int kPitch = kHeadDim + 8;        // 16-bit elements
    const float inv = __frcp_rn(l);     // a division for each output took a quarter of the kernel's instructions
    auto pair = [&](float e0, float e1) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(e0 * inv, e1 * inv);
        return *reinterpret_cast<const uint32_t *>(&r);
    };
    uint32_t probe = 0u;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
        const uint2 y = make_uint2(pair(sum[i].x, sum[i].y), pair(sum[i].z, sum[i].w));
        *reinterpret_cast<uint2 *>(rows + mine * kPitch + 4 * (quad + i)) = y;
        probe = probe_finite(y.y, probe_finite(y.x, probe));
    }
    // 8-bit values are finite or NaN, which any weight gives
    if (!E4M3 && __builtin_expect(bf16x2_nonfinite(probe) && l > 0.f, 0))
        put_seen_nonfinite(a, j, row0 + nth, quad, kQuads, rows + mine * kPitch + 4 * quad);
    __syncthreads();
    constexpr int kChunks = 16 / SPLIT;     // of 16 bytes
    for (int i = threadIdx.x; i < here * g * kChunks; i += kJoinThreads) {
        const int v = i / kChunks, c = i % kChunks + blockIdx.z * kChunks, at = v / g;
        *reinterpret_cast<uint4 *>(a.out + (size_t)(row0 + at) * a.ldo + (size_t)(j * g + v - at * g) * kHeadDim + 8 * c) =
            *reinterpret_cast<const uint4 *>(rows + v * kPitch + 8 * c);
    }
}

// Innermost first: half an entry's elements, entries, (sequence, head), halves: a tile's two halves in one copy.  The cache
// is stored with its 16-byte chunks already permuted by position, as the
// 128-byte swizzle wants them in shared memory (parts and tiles start at multiples of 8), so the copy
// permutes nothing.
bool encode_cache(CUtensorMap *m, const void *base, int rows, int max_len, int outer, const char **why) {
    return encode_tiles<4>(m, base, {64, cuuint64_t(rows), cuuint64_t(outer), 2},
                           {cuuint64_t(kHeadDim) * 2, cuuint64_t(max_len) * kHeadDim * 2, 128}, {64, kKeys, 1, 2},
                           CU_TENSOR_MAP_SWIZZLE_NONE, why);
}

}  // namespace

// Workspace: the status block, whose byte 128 is the item counter, then the lane
// GEMM's split-K counters, not used here, then the results.  No operator
// has scratch in the status block, so the counter is zero whatever a workspace
// was used for before, and a GEMM that uses it next finds its counters as it left them.
constexpr size_t kCounterAt = 128, kResultsAt = 256 + kCounterBytes;

size_t attn_tree_bytes(const KvBatch &own, int prefix_len, int group, int n) {
    const Plan p = plan_of(own, prefix_len, group, n, 1);
    return kResultsAt + size_t(slots_of(p, own.n_kv, group)) * (kHeadDim * sizeof(float) + sizeof(float2)) +
           expanded_bytes(p, prefix_len, own.n_kv);
}

namespace {

// The attention kernel over the prefix's parts, own parts or both.
template <bool E4M3>
cudaError_t launch_parts(KernelArgs &k, bool prefix, bool own, bool overlaps, cudaStream_t s) {
    static std::atomic<bool> opted_in[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !opted_in[dev]) {
        e = cudaFuncSetAttribute(attn_tree_kernel<E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemBytes<E4M3>));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) opted_in[dev] = true;
    }
    const KvBatch &c = k.a.own;
    k.prefix_parts = prefix ? k.p.n_parts : 0;
    k.own_parts = own;
    k.overlaps = overlaps;
    const long long items = (long long)c.n_kv * ((long long)k.prefix_parts * k.p.pairs +
                                                 (own ? (long long)c.n_seq * k.p.own_parts_max * k.p.own_pairs : 0));
    const int sms = device_sm_count();
    return launch_pdl(attn_tree_kernel<E4M3>, dim3(unsigned(items < sms ? items : sms)), dim3(Form<E4M3>::threads), kSmemBytes<E4M3>,
                      s, k);
}

template <bool E4M3>
cudaError_t launch_join(const KernelArgs &k, cudaStream_t s) {
    static std::atomic<bool> opted_in[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !opted_in[dev]) {
        for (const auto kernel : {attn_tree_join_kernel<E4M3, 32, 4, 2>, attn_tree_join_kernel<E4M3, 32, 1, 2>, attn_tree_join_kernel<E4M3, 32, 1, 3>})
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(JoinShared<32>)));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) opted_in[dev] = true;
    }
    const AttnTreeArgs &a = k.a;
    // Vectors of a CTA of the sum: no more than 16 nodes, two a warp (64 x 64 nodes of one head, 8 vectors: 22 us in all, 32: 26;
    // 40 x 20 of three, 8: 28, 32: 21).  Columns split where there are fewer CTAs than kSplitCtas
    // (3 x 41 nodes, 84 CTAs, over own 12007 entries: 31 us, 41 without; 5 x 24, 240 CTAs: 52, 41 without; few parts gain
    // nothing: 8 nodes over 300 entries 11.1, 10.1 without).
    // Three CTAs an SM, with half the loads on their way, from kFullCtas on (24 x 64 nodes of 8 heads: 1,074 us, 1,086 with
    // two; 64 x 64 over 500 entries 225, 254 with two; 5 x 24: 43, 41 with two).
    constexpr int kSplitCtas = 100, kFullCtas = 456;
    const int vecs = a.group == 1 ? 8 : 32, nodes = vecs / a.group, ctas = (k.p.rows + nodes - 1) / nodes * a.own.n_kv;
    auto join = [&](auto kernel, int split, size_t smem) {
        return launch_pdl(kernel, dim3(ctas / a.own.n_kv, a.own.n_kv, split), dim3(kJoinThreads), smem, s, a, k.p,
                          (const float *)k.values, (const float2 *)k.ml, k.next);
    };
    if (vecs == 8) return join(attn_tree_join_kernel<E4M3, 8, 1, 2>, 1, sizeof(JoinShared<8>));
    if (ctas < kSplitCtas) return join(attn_tree_join_kernel<E4M3, 32, 4, 2>, 4, sizeof(JoinShared<32>));
    if (ctas < kFullCtas) return join(attn_tree_join_kernel<E4M3, 32, 1, 2>, 1, sizeof(JoinShared<32>));
    return join(attn_tree_join_kernel<E4M3, 32, 1, 3>, 1, sizeof(JoinShared<32>));
}

}  // namespace

cudaError_t launch_attn_tree(const AttnTreeArgs &a, cudaStream_t s, const char **why) {
    KernelArgs k{};
    k.a = a;
    const int sms = device_sm_count();
    k.p = plan_of(a.own, a.prefix_len, a.group, a.n, sms > 0 ? sms : 1);
    char *base = static_cast<char *>(a.ws);
    k.next = reinterpret_cast<unsigned *>(base + kCounterAt);
    const size_t slots = size_t(slots_of(k.p, a.own.n_kv, a.group));
    char *const expanded = base + kResultsAt;
    const size_t half = expanded_bytes(k.p, a.prefix_len, a.own.n_kv) / 2;
    k.values = reinterpret_cast<float *>(expanded + 2 * half);
    k.ml = reinterpret_cast<float2 *>(k.values + slots * kHeadDim);
    const bool e4m3 = a.own.format == kKvE4m3;
    bool ok = encode_queries(&k.map[4], a.q, a.own.n_kv * a.group, k.p.rows, a.ldq, a.group, k.p.rows_tile, why);
    if (a.prefix_len > 0 && (!e4m3 || k.p.expanded)) {
        const void *pk = e4m3 ? expanded : a.prefix.k, *pv = e4m3 ? expanded + half : a.prefix.v;
        const int len = e4m3 ? expanded_len(a.prefix_len) : a.prefix.max_len;
        ok = ok && encode_cache(&k.map[0], pk, a.prefix_len, len, a.own.n_kv, why) &&
             encode_cache(&k.map[1], pv, a.prefix_len, len, a.own.n_kv, why);
    }
    if (!e4m3)
        ok = ok && encode_cache(&k.map[2], a.own.k, a.own.max_len, a.own.max_len, a.own.n_seq * a.own.n_kv, why) &&
             encode_cache(&k.map[3], a.own.v, a.own.max_len, a.own.max_len, a.own.n_seq * a.own.n_kv, why);
    if (!ok) return cudaErrorInvalidValue;
    cudaError_t e;
    if (k.p.expanded) {
        const dim3 grid((a.prefix_len + kExpandEntries - 1) / kExpandEntries, a.own.n_kv, 2);
        e = launch_pdl(expand_prefix_kernel, grid, dim3(256), 0, s, a.prefix, a.prefix_len, expanded_len(a.prefix_len),
                       reinterpret_cast<uint4 *>(expanded), reinterpret_cast<uint4 *>(expanded + half));
        if (e == cudaSuccess) e = launch_parts<false>(k, true, false, false, s);
        if (e == cudaSuccess) {
            ++k.next;       // each grid has its counter
            e = launch_parts<true>(k, false, true, true, s);
            --k.next;
        }
    } else {
        e = e4m3 ? launch_parts<true>(k, true, true, false, s) : launch_parts<false>(k, true, true, false, s);
    }
    if (e != cudaSuccess) return e;
    return e4m3 ? launch_join<true>(k, s) : launch_join<false>(k, s);
}

}  // namespace tfk
