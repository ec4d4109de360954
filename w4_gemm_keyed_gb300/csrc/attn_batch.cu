// Attention of a batch of sequences that continue one prompt.
//
// Row r of sequence b (position pos[b] + r of its own cache) attends over the
// shared prefix's entries 0 .. P - 1 and its own entries 0 .. pos[b] + r:
//   s_t = q . k_t / sqrt(128),  o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m).
//
// Keys are cut into parts: the prefix into parts of a length that depends on P
// and the number of KV heads only, each sequence's own entries into parts of
// kOwnPart.  An item is one part of one KV head with the query vectors that
// read it: for a prefix part, up to 256 of the batch's n_seq * R * group vectors
// (the prefix is read once for all of them, from HBM once and from L2 for the
// rest), for an own part the sequence's R * group.  Within an item each vector
// folds its keys in ascending order, 128 at a time, with a running maximum; the
// parts' results (maximum m, weight sum l, unnormalised output o, fp32) are
// joined per vector in ascending order by a second kernel.  So a row's bits
// depend on its query, its position, P and the entries it sees alone:
// matrix-product rows never mix, and keys past a row's last add exact zeros.
//
// Scores and outputs run on tcgen05 with 128 query vectors as M: S = Q K^T with
// both operands in shared memory and S in tensor memory, then P (bf16, in place
// of S) times V with P read from tensor memory.  A tile of 128 vectors is filled
// by rows x group; with few of them the rest are idle, and a 128-key tile still
// takes an SM about 2,000 cycles where HBM delivers one (K and V) to each SM in
// 2,800, so few rows need no form of their own.
//
// What bounds it (GB300, measured call after call on the same inputs): many rows, the
// tensor cores and the hand-over between them and the softmax: a step of two tiles and
// 128 keys takes about 2,700 cycles where its products take 2,080 (512 rows x 64 heads over
// 32768 entries 424 us, 1.29 PFLOP/s; 444 to 448 with other inputs each call; of that the
// steps about 300, passing from item to item 42, joining about 47).  Few rows, HBM: 12 rows
// x 20 heads over 130001 entries 51 us, 5.2 TB/s.  E4M3 caches with many rows, the chain
// of hand-overs that expanding each tile makes longer, with no unit near its limit (issue
// 45 %, ALU 34 %, tensor 33 %, shared memory 19 %): 240 rows x 64 heads over 20000
// entries 212 us, 169 as a bf16 cache.
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn_batch.cuh"
#include "tf_tcgen05.cuh"
#include "w4_gemm.cuh"

namespace tfk {

namespace {

constexpr float kScaleLog2 = 0.12751743074439720f;   // log2(e) / sqrt(128)
// A vector's reference maximum moves only when a score passes it by more than
// 2^8 in weight: weights stay below 2^8 (exact in the sums' exponents), and the
// output is rescaled rarely.  The decision is the vector's own.
constexpr float kMaxSlack = 8.0f / kScaleLog2;

constexpr int kTile = 128;              // query vectors and keys per matrix product
constexpr int kOwnPart = 512;           // own entries per part
constexpr int kMinPrefixPart = 512;     // shared entries per part, at least
constexpr int kHalfBytes = kTile * 128; // 64 elements of 128 rows
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr int kRing = 4;                // items known ahead
constexpr int kGroups = 256;            // entries of the table of own parts
constexpr int kSoftmaxWarps = 8, kProducerWarp = 8, kMmaWarp = 9;
constexpr int kExpandWarp = 12, kExpandWarps = 8;

// What the cache's format changes: an E4M3 tile (16 KB and 128 scale bytes) is
// copied into a raw stage and expanded by eight more warps into a bf16 tile, so
// the products are those of a bf16 cache holding the same values.
template <bool E4M3>
struct Form {
    static constexpr int stages = E4M3 ? 3 : 5;         // bf16 K and V tiles in shared memory
    // E4M3 tiles on their way (4 expanded + 2 raw: 0.7 % slower at 240 rows over 20000 entries,
    // 2 % at 12 rows over 130001; 3 + 4 as 3 + 3)
    static constexpr int raw = E4M3 ? 3 : 0;
    static constexpr int threads = E4M3 ? 640 : 384;
    static constexpr int readers = kSoftmaxWarps + 1 + (E4M3 ? kExpandWarps : 0);  // of the item ring
    // registers a thread: the softmax warps' and the others', together no more
    // than the launch's share (96 a thread of 640, 168 of 384).  With 144 and 64 (240 E4M3
    // rows), 208 and 88 (512 bf16 rows): 0.5 % and 1 % slower.
    static constexpr int regs_softmax = E4M3 ? 168 : 216, regs_other = E4M3 ? 48 : 72;
    static_assert(256 * regs_softmax + (threads - 256) * regs_other <= threads * (E4M3 ? 96 : 168), "register split");
};
constexpr int kRawBytes = kTile * kHeadDim;
constexpr uint32_t kTmemCols = 512, kTmemS = 0, kTmemO = 256;

struct Item {
    int n_vec;          // query vectors (0: no more items)
    int n_keys;         // entries of the part
    int j, b;           // KV head, sequence (-1: prefix)
    int vec0;           // first vector: (row * group + head) within KV head j
    int key0;           // first entry
    int lim0;           // part entry index of row 0's last visible entry (own), n_keys - 1 (prefix)
    int stride;         // vectors per column quad of the partial output
    long long part;     // index of the part's first (vector, column quad 0) in opart / 32, and in ml
};

// Prefix partials: [part][n_kv][tiles][32 quads][tile vectors][4]; own partials:
// [part][n_seq][n_kv][32 quads][R * group][4].  Maxima and sums: the same
// without the quads.  Quad-major so that a warp's 32 vectors store and load 512
// consecutive bytes.
struct Plan {
    int n_vec, tile, tiles, pairs;      // vectors; per tile; tiles and pairs of them per KV head
    int part, n_parts;          // prefix part length and count
    int own_parts_max;
    long long own0;             // index of the first own vector slot after the prefix's
    long long slots;            // vector slots in all
};

__host__ __device__ inline int prefix_part(int prefix_len, int n_kv) {
    // Parts that make about kItems items where the batch is a single tile, none
    // shorter than kMinPrefixPart.  Few rows want many parts (each SM streams one),
    // many rows few (each is stored and joined per vector).  12 rows over 130001
    // entries / 512 rows over 32768, 4 and 8 heads, against 100 items with kernels slower
    // than these: 152 items 2 % / 5 % slower, 76 items 20 % slower / 2 % faster.
    constexpr int kItems = 100;
    const long long even = ((long long)prefix_len * n_kv + kItems - 1) / kItems;
    const long long part = (even + kTile - 1) / kTile * kTile;
    return int(part < kMinPrefixPart ? kMinPrefixPart : part);
}

Plan plan_of(const KvBatch &own, int prefix_len, int group, int R) {
    Plan p;
    p.n_vec = own.n_seq * R * group;
    p.tile = kTile / group * group;     // whole rows, so that a tile of queries is one box to TMA
    p.tiles = (p.n_vec + p.tile - 1) / p.tile;
    p.pairs = (p.tiles + 1) / 2;
    p.part = prefix_part(prefix_len, own.n_kv);
    p.n_parts = (prefix_len + p.part - 1) / p.part;
    p.own_parts_max = (own.max_len + kOwnPart - 1) / kOwnPart;
    p.own0 = (long long)p.n_parts * own.n_kv * p.tiles * p.tile;
    p.slots = p.own0 + (long long)p.own_parts_max * own.n_kv * p.n_vec;
    return p;
}

struct KernelArgs {
    CUtensorMap map[5];     // prefix K, V; own K, V (bf16 caches); queries
    AttnBatchArgs a;
    Plan p;
    float *opart;           // [slots][128]
    float2 *ml;             // [slots]: (maximum score, weight sum)
    unsigned *next;         // items taken beyond the first of each CTA; zero between calls
};

// A parity wait tells a phase from its neighbours only, so whoever waits on a
// barrier waits on every one of its phases, and before the next can end.  Hence three barriers for scores:
// S0 and S1 of one-tile items and S0 of two-tile items are read by the first
// softmax group (0, 1, 0), S1 of two-tile items by the second (2).
struct __align__(16) Shared {
    uint64_t kv_full[5], kv_empty[5], raw_full[3], raw_empty[3];
    uint64_t q_full[2], q_empty[2], s_full[3], p_full[2][2], o_done[2];
    uint64_t item_full[kRing], item_empty[kRing], drain;
    Item item[kRing];
    unsigned before[kGroups + 1];   // own parts of the sequence groups before each
    uint32_t tmem;
    int abort;
};
// query tiles, bf16 stages, raw stages, their scales, then Shared
template <bool E4M3>
constexpr size_t kSmemBytes = size_t(2 + Form<E4M3>::stages) * kTileBytes + size_t(Form<E4M3>::raw) * (kRawBytes + kTile) +
                              sizeof(Shared);
static_assert(kSmemBytes<false> <= 227 * 1024 && kSmemBytes<true> <= 227 * 1024, "shared memory");

template <int N>
__device__ __forceinline__ void regs_raise() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_lower() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A wait of one thread that is its warp's only one in the role.
__device__ __forceinline__ bool lane_wait(Shared *sh, uint64_t *bar, uint32_t parity) {
    return mbar_wait_or_abort(&sh->abort, bar, parity);
}

// A wait of a converged warp: all lanes get one answer, so that they go on or end the
// role together, and leave it converged, as what follows requires (shuffles, votes,
// tensor memory).  The vote costs 240 rows over E4M3 entries 2 % (208 to 213 us), 512
// rows over bf16 ones 0.6 %.
__device__ __forceinline__ bool warp_wait(Shared *sh, uint64_t *bar, uint32_t parity) {
    return mbar_warp_wait_or_abort(&sh->abort, bar, parity);
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

__device__ __forceinline__ bool bf16x2_nonfinite(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ uint32_t bf16x2_finite(uint32_t w) {   // non-finite halves -> 0
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
    return w;
}

// ------------------------------------------------------------------ item order
// Prefix items first (the longest), vector pairs fastest so that the CTAs working
// on one part read it from L2; then own items, heads fastest.
__device__ int own_parts(const KernelArgs &k, int b, bool report) {
    const long long p = seq_position(k.a.pos, b, k.a.R, k.a.own.max_len, k.a.err, report);
    return p < 0 ? 0 : int((p + k.a.R - 1) / kOwnPart) + 1;
}

__device__ Item item_of(const KernelArgs &k, const Shared *sh, unsigned i, int group_seqs) {
    Item it{};
    const unsigned n_kv = k.a.own.n_kv, rg = k.a.R * k.a.group, pairs = k.p.pairs;
    const unsigned n_prefix = k.p.n_parts * n_kv * pairs;
    if (i < n_prefix) {
        const unsigned cj = idx_div(i, pairs), pair = i - cj * pairs, c = idx_div(cj, n_kv);
        it.j = cj - c * n_kv;
        it.b = -1;
        it.vec0 = pair * 2 * k.p.tile;
        it.n_vec = min(2 * k.p.tile, k.p.n_vec - it.vec0);
        it.key0 = c * k.p.part;
        it.n_keys = min(k.p.part, k.a.prefix_len - it.key0);
        it.lim0 = it.n_keys - 1;
        it.stride = k.p.tile;
        it.part = ((long long)cj * k.p.tiles + 2 * pair) * k.p.tile;
        return it;
    }
    i -= n_prefix;
    const int n_groups = (k.a.own.n_seq + group_seqs - 1) / group_seqs;
    if (i >= sh->before[n_groups] * n_kv) return it;
    int u = idx_div(i, n_kv);
    it.j = i - u * n_kv;
    int lo = 0, hi = n_groups - 1;      // last group whose parts start at or before u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sh->before[mid] <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    u -= sh->before[lo];
    int b = lo * group_seqs;
    for (int n; u >= (n = own_parts(k, b, false)); ++b) u -= n;
    const long long p = k.a.pos[b];
    it.b = b;
    it.vec0 = b * rg;
    it.n_vec = rg;
    it.key0 = u * kOwnPart;
    it.n_keys = int(min((long long)kOwnPart, p + k.a.R - it.key0));
    it.lim0 = int(p - it.key0);
    it.stride = rg;
    it.part = k.p.own0 + (((long long)u * k.a.own.n_seq + b) * n_kv + it.j) * rg;
    return it;
}

// ------------------------------------------------------------------ roles
// One CTA per SM takes items from a common counter.
//   warp 8      finds the next item and streams its query vectors and its K and V
//               tiles by TMA
//   warp 9      issues the products
//   warps 12-19 expand E4M3 tiles (there alone)
//   warps 0-7   softmax: a thread per vector.  Items of two tiles give one tile to
//               each group of four warps; items of one tile use the second tile's
//               S columns so that the next key tile's scores are computed
//               while this one's are being exponentiated.

template <bool E4M3>
__device__ void produce(const KernelArgs &k, Shared *sh, uint8_t *q_tiles, uint8_t *stages) {
    constexpr int kStages = E4M3 ? Form<E4M3>::raw : Form<E4M3>::stages;
    uint64_t *const full = E4M3 ? sh->raw_full : sh->kv_full, *const empty = E4M3 ? sh->raw_empty : sh->kv_empty;
    const int lane = threadIdx.x & 31, n_seq = k.a.own.n_seq;
    const int group_seqs = (n_seq + kGroups - 1) / kGroups;
    const int n_groups = (n_seq + group_seqs - 1) / group_seqs;
    int total = 0;
    for (int g0 = 0; g0 < n_groups; g0 += 32) {
        int n = 0;
        for (int b = (g0 + lane) * group_seqs; b < min(n_seq, (g0 + lane + 1) * group_seqs); ++b)
            n += own_parts(k, b, blockIdx.x == 0);
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
    if (lane != 0) return;

    unsigned i = blockIdx.x;
    unsigned loaded = 0;     // K and V tiles so far
    unsigned q_uses[2] = {0, 0};
    int q_next = 0;          // the query tile of the next one-tile item
    const int g = k.a.group;
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (n >= kRing && !lane_wait(sh, &sh->item_empty[slot], (n / kRing - 1) & 1)) break;
        const Item it = item_of(k, sh, i, group_seqs);
        sh->item[slot] = it;
        mbar_arrive(&sh->item_full[slot]);
        const unsigned taken = atomicAdd(k.next, 1u);       // the item after this one
        if (it.n_vec == 0) break;
        const bool own = it.b >= 0;
        const int tiles = (it.n_keys + kTile - 1) / kTile, outer = own ? it.b * k.a.own.n_kv + it.j : it.j;
        const void *map_k = &k.map[own ? 2 : 0], *map_v = &k.map[own ? 3 : 1];
        bool ok = true;
        // Queries first: behind the next item's K and V tiles they came 5,400 cycles late.
        // A tile is whole rows of the KV head's query heads, one box of (64 elements,
        // heads, rows) per half, swizzled into a K-major tile.  Rows of the box past
        // the item's (another sequence's, or zeros past the last) fill vectors that
        // nothing reads: rows of a product never mix.
        const bool two = it.n_vec > k.p.tile;
        for (int t = 0; t < (two ? 2 : 1) && ok; ++t) {
            const int buf = two ? t : q_next;
            if (q_uses[buf] > 0) ok = lane_wait(sh, &sh->q_empty[buf], (q_uses[buf] - 1) & 1);
            if (!ok) break;
            ++q_uses[buf];
            const int row = (it.vec0 + t * k.p.tile) / g;
            mbar_arrive_expect_tx(&sh->q_full[buf], 2 * uint32_t(k.p.tile) * 128u);
            tma_load_3d(q_tiles + buf * kTileBytes, &k.map[4], 0, it.j * g, row, &sh->q_full[buf]);
            tma_load_3d(q_tiles + buf * kTileBytes + kHalfBytes, &k.map[4], 64, it.j * g, row, &sh->q_full[buf]);
        }
        if (!two) q_next ^= 1;
        for (int t = 0; t < 2 * tiles && ok; ++t, ++loaded) {
            const bool is_v = order_is_v(t, tiles);
            const int row = it.key0 + order_tile(t, tiles) * kTile;
            const int st = loaded % kStages;
            if (loaded >= kStages) ok = lane_wait(sh, &empty[st], (loaded / kStages - 1) & 1);
            if (!ok) break;
            if constexpr (E4M3) {
                const KvBatch &c = own ? k.a.own : k.a.prefix;
                const uint32_t rows = uint32_t(min(kTile, it.key0 + it.n_keys - row)), scales = (rows + 15u) & ~15u;
                const size_t entry = (size_t)outer * c.max_len + (size_t)row;
                uint8_t *dst = stages + size_t(st) * kRawBytes;
                mbar_arrive_expect_tx(&full[st], rows * kHeadDim + scales);
                bulk_g2s(dst, static_cast<const uint8_t *>(is_v ? c.v : c.k) + entry * kHeadDim, rows * kHeadDim, &full[st]);
                bulk_g2s(stages + size_t(kStages) * kRawBytes + st * kTile, (is_v ? c.v_scale : c.k_scale) + entry, scales,
                         &full[st]);
            } else {
                uint8_t *dst = stages + size_t(st) * kTileBytes;
                mbar_arrive_expect_tx(&full[st], kTileBytes);
                tma_load_3d(dst, is_v ? map_v : map_k, 0, row, outer, &full[st]);
                tma_load_3d(dst + kHalfBytes, is_v ? map_v : map_k, 64, row, outer, &full[st]);
            }
        }
        if (!ok) break;
        i = gridDim.x + taken;
    }
    // no copy outlives the CTA
    for (unsigned t = loaded > kStages ? loaded - kStages : 0; t < loaded; ++t)
        wait_drained(&full[t % kStages], (t / kStages) & 1);
    for (int buf = 0; buf < 2; ++buf)
        if (q_uses[buf] > 0) wait_drained(&sh->q_full[buf], (q_uses[buf] - 1) & 1);
}

// E4M3 tiles -> bf16 tiles, eight lanes an entry.  Rows of a V tile past the
// part's last entry become zeros up to the 16-row step the product reads, and so
// do entries marked NaN that some rows do not see (0 * NaN would reach those
// rows; the rows that see them get the NaN back when the output is stored).
__device__ void expand_tiles(const KernelArgs &k, Shared *sh, uint8_t *stages, const uint8_t *raw) {
    constexpr int kStages = Form<true>::stages, kRaw = Form<true>::raw;
    const int lane = threadIdx.x & 31, tid = threadIdx.x - 32 * kExpandWarp, group = tid & 7;
    const uint8_t *scales = raw + size_t(kRaw) * kRawBytes;
    unsigned done = 0;
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (!warp_wait(sh, &sh->item_full[slot], (n / kRing) & 1)) return;
        const Item it = sh->item[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
        if (it.n_vec == 0) return;
        const int tiles = (it.n_keys + kTile - 1) / kTile;
        for (int t = 0; t < 2 * tiles; ++t, ++done) {
            const bool is_v = order_is_v(t, tiles);
            const int key = order_tile(t, tiles) * kTile, valid = min(kTile, it.n_keys - key);
            const int fill = is_v ? (valid + 15) & ~15 : valid, hidden = it.lim0 + 1 - key;
            const int rs = done % kRaw, st = done % kStages;
            if (!warp_wait(sh, &sh->raw_full[rs], (done / kRaw) & 1)) return;
            if (done >= kStages && !warp_wait(sh, &sh->kv_empty[st], (done / kStages - 1) & 1)) return;
            constexpr int kRows = 4 * kExpandWarps, kSteps = kTile / kRows;    // rows all warps take at a time
            static_assert(kRows % 8 == 0 && kTile % kRows == 0, "a thread's rows share their place in the swizzle");
            const int row0 = tid >> 3;
            const uint8_t *src = raw + size_t(rs) * kRawBytes + row0 * kHeadDim + 16 * group;
            const uint8_t *sc = scales + rs * kTile + row0;
            uint8_t *dst = stages + size_t(st) * kTileBytes + row0 * 128 + ((group ^ (row0 & 7)) << 4);
            const bool whole = valid == kTile && !(is_v && hidden < kTile);     // nothing to leave out
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
                *reinterpret_cast<uint4 *>(dst + i * kRows * 128 + kHalfBytes) = hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh->kv_full[st]);
                mbar_arrive(&sh->raw_empty[rs]);
            }
        }
    }
}

// The last V tiles of an own part: rows past the sequence's last entry become
// zeros (up to the 16-row step the product reads), and non-finite elements of
// entries that some rows do not see become zero, since 0 * inf would reach
// those rows; the rows that see them get them back when the output is stored.
__device__ __forceinline__ void mend_values(uint8_t *v, int first_hidden, int valid, int lane) {
    const int end = (valid + 15) & ~15;
    for (int i = first_hidden * 16 + lane; i < end * 16; i += 32) {
        const int row = i >> 4, c = i & 15;
        uint4 *p = reinterpret_cast<uint4 *>(v + (c >> 3) * kHalfBytes + row * 128 + (((c & 7) ^ (row & 7)) << 4));
        if (row >= valid) {
            *p = make_uint4(0u, 0u, 0u, 0u);
        } else {
            const uint4 x = *p;
            if (bf16x2_nonfinite(x.x) || bf16x2_nonfinite(x.y) || bf16x2_nonfinite(x.z) || bf16x2_nonfinite(x.w))
                *p = make_uint4(bf16x2_finite(x.x), bf16x2_finite(x.y), bf16x2_finite(x.z), bf16x2_finite(x.w));
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// The whole warp follows the items; the elected lane waits, issues and commits, so
// that nothing but those is on the products' path (with every lane in every wait
// and a predicate on each product, the call took 8 % longer at 512 rows over 32768 entries).
template <bool E4M3>
__device__ void multiply(const KernelArgs &k, Shared *sh, uint8_t *q_tiles, uint8_t *stages, uint32_t tmem) {
    constexpr int kStages = Form<E4M3>::stages;
    const int lane = threadIdx.x & 31;
    const bool leader = elect_one() != 0;
    unsigned taken = 0;                  // K and V tiles of the items before this one
    unsigned q_uses[2] = {0, 0}, p_uses[2] = {0, 0};
    int next = 0;
    const uint32_t q_addr = smem_u32(q_tiles), st_addr = smem_u32(stages);

    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (!warp_wait(sh, &sh->item_full[slot], (n / kRing) & 1)) break;
        // broadcast: the same in all lanes, and known to be
        const int n_vec = __shfl_sync(0xFFFFFFFFu, sh->item[slot].n_vec, 0);
        const int n_keys = __shfl_sync(0xFFFFFFFFu, sh->item[slot].n_keys, 0);
        const int lim0 = __shfl_sync(0xFFFFFFFFu, sh->item[slot].lim0, 0);
        const int seq = __shfl_sync(0xFFFFFFFFu, sh->item[slot].b, 0);
        if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
        __syncwarp();
        if (n_vec == 0) break;
        const bool two = n_vec > k.p.tile;
        const int tiles = (n_keys + kTile - 1) / kTile;
        const int q0 = two ? 0 : next;
        auto stage_of = [&](int order) { return (taken + order) % kStages; };
        auto wait_tile = [&](int order) {
            return lane_wait(sh, &sh->kv_full[stage_of(order)], ((taken + order) / kStages) & 1);
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
        }
        // own parts end in V tiles to mend, which takes the whole warp
        const int whole = E4M3 || seq < 0 ? tiles : min(tiles, max(0, (lim0 + 1) / kTile));
        if (leader)
            for (int i = 0; i < whole && ok; ++i) ok = step(i);
        __syncwarp();
        for (int i = whole; i < tiles; ++i) {
            if (!warp_wait(sh, &sh->kv_full[stage_of(v_order(i, tiles))], ((taken + v_order(i, tiles)) / kStages) & 1)) {
                ok = false;
                break;
            }
            const int keys = min(kTile, n_keys - i * kTile), hidden = max(0, lim0 + 1 - i * kTile);
            mend_values(stages + stage_of(v_order(i, tiles)) * size_t(kTileBytes), min(hidden, keys), keys, lane);
            if (leader) ok = ok && step(i);
            __syncwarp();
        }
        if (__any_sync(0xFFFFFFFFu, !ok)) break;
        taken += 2 * tiles;
        if (!two) next ^= 1;
    }
    // no product outlives the CTA, whichever way the loop ended
    if (leader) {
        tc_commit(&sh->drain);
        wait_drained(&sh->drain, 0);
    }
    __syncwarp();
}

// Rows that see an own entry with non-finite values get them back: mend_values
// took them out of the product.  x: one element of the output, d its index.
template <bool E4M3>
__device__ __forceinline__ float with_nonfinite(const KernelArgs &k, const Item &it, int first, int last, int d, float x) {
    for (int t = first; t <= last; ++t) {
        const long long pos = (long long)it.key0 + t;
        const size_t entry = ((size_t)it.b * k.a.own.n_kv + it.j) * k.a.own.max_len + (size_t)pos;
        if constexpr (E4M3) {
            if (k.a.own.v_scale[entry] == kScaleNan) x = __uint_as_float(0x7FC00000u);
        } else {
            const uint16_t v =
                static_cast<const uint16_t *>(k.a.own.v)[entry * kHeadDim + 8 * ((d >> 3) ^ int(pos & 7)) + (d & 7)];
            if ((v & 0x7F80u) == 0x7F80u) x += __uint_as_float(uint32_t(v) << 16);
        }
    }
    return x;
}

// Whether any value of the part's entries first .. last (at most 15) is not finite; whole warp.
template <bool E4M3>
__device__ __forceinline__ bool any_nonfinite(const KernelArgs &k, const Item &it, int first, int last, int lane) {
    bool bad = false;
    if constexpr (E4M3) {
        if (first + lane <= last)
            bad = k.a.own.v_scale[((size_t)it.b * k.a.own.n_kv + it.j) * k.a.own.max_len + (size_t)(it.key0 + first + lane)] ==
                  kScaleNan;
    } else {
        for (int i = first * 16 + lane; i < (last + 1) * 16; i += 32) {
            const size_t entry = ((size_t)it.b * k.a.own.n_kv + it.j) * k.a.own.max_len + (size_t)(it.key0 + (i >> 4));
            const uint4 x =
                *(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(k.a.own.v) + entry * kHeadDim) + (i & 15));
            bad |= bf16x2_nonfinite(x.x) || bf16x2_nonfinite(x.y) || bf16x2_nonfinite(x.z) || bf16x2_nonfinite(x.w);
        }
    }
    return __any_sync(0xFFFFFFFFu, bad);
}

template <bool E4M3>
__device__ void softmax(const KernelArgs &k, Shared *sh, uint32_t tmem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wg = warp >> 2;
    const uint32_t my_lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t t_o = tmem + kTmemO + wg * kHeadDim + my_lanes;
    unsigned s_uses[2] = {0, 0}, o_uses = 0;     // the second group counts its barrier in s_uses[1]
    for (unsigned n = 0;; ++n) {
        const int slot = n % kRing;
        if (!warp_wait(sh, &sh->item_full[slot], (n / kRing) & 1)) return;
        const Item &it = sh->item[slot];        // read where it is needed: registers are short
        if (it.n_vec == 0) return;
        auto release = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
        };
        const bool two = it.n_vec > k.p.tile;
        const int tiles = (it.n_keys + kTile - 1) / kTile;
        if (wg == 1 && !two) {
            release();
            continue;
        }
        const int v = 32 * (warp & 3) + lane;               // vector within the tile
        const int n_here = min(k.p.tile, it.n_vec - wg * k.p.tile);     // of this tile
        const bool active = 32 * (warp & 3) < n_here;
        const int lim = it.b < 0 ? it.lim0 : it.lim0 + min(v, it.n_vec - 1) / k.a.group;     // last visible part entry
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < tiles; ++i) {
            const int buf = two ? wg : i & 1;
            if (!warp_wait(sh, &sh->s_full[wg ? 2 : buf], s_uses[buf]++ & 1)) return;
            bool seen = i == 0;     // whether the previous tile's product into the output is known to be done
            if (active) {
                tc_fence_after();
                const uint32_t t_s = tmem + kTmemS + buf * kTile + my_lanes;
                const int last = lim - i * kTile;
                const bool part_seen = __any_sync(0xFFFFFFFFu, last < kTile - 1);
                // bf16 caches: all scores in registers (512 rows over 32768 entries: 5 % slower with
                // the upper half read again for its weights, as below).  The softmax of
                // E4M3 caches has fewer: 64 scores at a time, the upper half for its maximum
                // first, and once more after the lower half's weights have been stored; its
                // loops stay rolled, as instructions are fetched anew for every role between.
                uint32_t x[64], y[E4M3 ? 1 : 64];
                float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto fetch = [&](int c0, uint32_t *s) {
                    tc_ld32(t_s + c0, s);
                    tc_ld32(t_s + c0 + 32, s + 32);
                };
                auto settle = [&](int c0, uint32_t *s) {    // after tc_wait_ld
                    tc_pin32(s);
                    tc_pin32(s + 32);
                    if (part_seen) {
#pragma unroll
                        for (int c = 0; c < 64; ++c) s[c] = c0 + c <= last ? s[c] : 0xFF800000u;
                    }
                };
                auto tops = [&](const uint32_t *s) {
#pragma unroll
                    for (int c = 0; c < 64; c += 2)
                        mt[(c >> 1) & 3] = max3(mt[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                };
                if constexpr (E4M3) {
#pragma unroll 1
                    for (int c0 = 64; c0 >= 0; c0 -= 64) {
                        fetch(c0, x);
                        tc_wait_ld();
                        settle(c0, x);
                        tops(x);
                    }
                } else {
                    fetch(0, x);
                    fetch(64, y);
                    tc_wait_ld();
                    settle(0, x);
                    settle(64, y);
                    tops(x);
                    tops(y);
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
                    if (h == 0) {       // the product with the first 64 keys may start
                        tc_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh->p_full[buf][0]);
                    }
                };
                if constexpr (E4M3) {
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        if (h == 1) {
                            fetch(64, x);
                            tc_wait_ld();
                            settle(64, x);
                        }
                        weigh(x, h);
                    }
                } else {
                    weigh(x, 0);
                    weigh(y, 1);
                }
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
        // entries that only some rows see
        const int first = max(0, it.lim0 + 1), end = it.n_keys - 1;
        const bool bad = active && it.b >= 0 && first <= end && any_nonfinite<E4M3>(k, it, first, end, lane);
        if (!warp_wait(sh, &sh->o_done[wg], (o_uses - 1) & 1)) return;
        if (!active) {
            release();
            continue;
        }
        tc_fence_after();
        const bool store = v < n_here;
        const long long part = it.part + (wg ? k.p.tile : 0);
        float4 *dst = reinterpret_cast<float4 *>(k.opart + part * kHeadDim) + v;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tc_ld32(t_o + 32 * c, o);
            tc_wait_ld();
            tc_pin32(o);
            if (store) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[(size_t)(8 * c + e) * it.stride] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                                       __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            }
        }
        if (store) k.ml[part + v] = make_float2(m, l);
        if (bad && store) {
            float *o = reinterpret_cast<float *>(dst);
            for (int d = 0; d < kHeadDim; ++d) {
                float *e = o + (size_t)(d >> 2) * it.stride * 4 + (d & 3);
                *e = with_nonfinite<E4M3>(k, it, first, min(lim, end), d, *e);
            }
        }
        tc_fence_before();      // the reads of O precede this warp's next arrival on p_full
        release();
    }
}

template <bool E4M3>
__global__ void __launch_bounds__(Form<E4M3>::threads, 1) attn_batch_kernel(const __grid_constant__ KernelArgs k) {
    using F = Form<E4M3>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_tiles = smem, *stages = smem + 2 * kTileBytes, *raw = stages + size_t(F::stages) * kTileBytes;
    Shared *sh = reinterpret_cast<Shared *>(raw + size_t(F::raw) * (kRawBytes + kTile));
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < F::stages; ++i) {
            mbar_init(&sh->kv_full[i], E4M3 ? kExpandWarps : 1);
            mbar_init(&sh->kv_empty[i], 1);
        }
        for (int i = 0; i < F::raw; ++i) {
            mbar_init(&sh->raw_full[i], 1);
            mbar_init(&sh->raw_empty[i], kExpandWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->q_full[i], 1);
            mbar_init(&sh->q_empty[i], 1);
            mbar_init(&sh->p_full[i][0], 4);
            mbar_init(&sh->p_full[i][1], 4);
            mbar_init(&sh->o_done[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh->item_full[i], 1);
            mbar_init(&sh->item_empty[i], F::readers);
        }
        for (int i = 0; i < 3; ++i) mbar_init(&sh->s_full[i], 1);
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tc_alloc(&sh->tmem, kTmemCols);
    if (warp == kProducerWarp && (threadIdx.x & 31) < 5 && (!E4M3 || (threadIdx.x & 31) == 4))
        prefetch_tensormap(&k.map[threadIdx.x & 31]);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    grid_dependency_wait();     // queries, positions and entries come from the preceding grids
    grid_launch_dependents();
    if (warp < kSoftmaxWarps) {
        regs_raise<F::regs_softmax>();
        softmax<E4M3>(k, sh, tmem);
    } else {
        regs_lower<F::regs_other>();
        if (warp == kProducerWarp)
            produce<E4M3>(k, sh, q_tiles, E4M3 ? raw : stages);
        else if (warp == kMmaWarp)
            multiply<E4M3>(k, sh, q_tiles, stages, tmem);
        else if (E4M3 && warp >= kExpandWarp)
            expand_tiles(k, sh, stages, raw);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && sh->abort) set_error(k.a.err, kDevTimeout);
    if (warp == kMmaWarp) tc_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ joining the parts
// A CTA takes 32 query vectors (lanes) and two column quads of one KV head; its
// four warps are four runs of consecutive parts.  A run's parts are folded in
// ascending order (prefix parts first) against the maximum of all the vector's
// parts, then the runs in ascending order: an order that the number of the vector's
// parts fixes.  Where there are many vectors, 520 bytes per vector and part from HBM
// or L2 and the instructions that find them bound it (with a quad a thread and 64-bit
// products for every part's place, 512 rows x 64 heads x 14 parts took 74 us, with
// two quads 55; CTAs of four quads, 256 threads, made the whole call 2 % slower than
// these); where there are few, the chain of three loads does.
constexpr int kJoinRuns = 4, kJoinUnroll = 4, kJoinThreads = 32 * kJoinRuns;

__global__ void __launch_bounds__(kJoinThreads, 6) attn_batch_join_kernel(AttnBatchArgs a, Plan p, const float *opart,
                                                                          const float2 *ml, unsigned *next) {
    __shared__ float s_top[kJoinRuns][32], s_l[kJoinRuns][32];
    __shared__ float4 s_o[kJoinRuns][2][32];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, quad = 2 * blockIdx.z;
    const int n_kv = a.own.n_kv, rg = a.R * a.group, j = blockIdx.y;
    const int v = blockIdx.x * 32 + lane;
    int n = 0, b = 0;
    if (v < p.n_vec) {
        b = idx_div(v, rg);
        const long long pos = seq_position(a.pos, b, a.R, a.own.max_len, a.err, false);
        if (pos >= 0) n = p.n_parts + int((pos + idx_div(v - b * rg, a.group)) / kOwnPart) + 1;
    }
    // Positions come from before the attention grid, which had waited for them when it
    // let this grid start; the partial results come from that grid itself.
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *next = 0u;
    const int c_begin = n * run / kJoinRuns, c_end = n * (run + 1) / kJoinRuns;
    // where a part's (maximum, sum) and values are: prefix parts, then own parts
    const int tile = idx_div(v, p.tile), in0 = v - tile * p.tile, in1 = v - b * rg;
    const size_t step0 = (size_t)n_kv * p.tiles * p.tile, step1 = (size_t)n_kv * p.n_vec;
    const size_t slot0 = (size_t)(j * p.tiles + tile) * p.tile, slot1 = (size_t)p.own0 + (size_t)(b * n_kv + j) * rg;
    const float4 *const values = reinterpret_cast<const float4 *>(opart);
    struct Place {
        const float2 *ml;
        const float4 *x;
    };
    const Place own = {ml + slot1 + in1, values + slot1 * 32 + quad * rg + in1};
    Place at;
    if (c_begin < p.n_parts)
        at = {ml + slot0 + c_begin * step0 + in0, values + (slot0 + c_begin * step0) * 32 + quad * p.tile + in0};
    else
        at = {own.ml + (c_begin - p.n_parts) * step1, own.x + (c_begin - p.n_parts) * step1 * 32};
    auto advance = [&](Place &q, int c) {       // from part c to part c + 1
        if (c + 1 == p.n_parts) {
            q = own;
        } else {
            const size_t step = c < p.n_parts ? step0 : step1;
            q.ml += step;
            q.x += step * 32;
        }
    };
    float2 w[kJoinUnroll];
    float4 x[kJoinUnroll][2];
    auto load = [&](int c) {        // parts c .. c + kJoinUnroll - 1 of this run
#pragma unroll
        for (int u = 0; u < kJoinUnroll; ++u) {
            w[u] = make_float2(-INFINITY, 0.f);
            if (c + u < c_end) {
                w[u] = *at.ml;
                x[u][0] = __ldcs(at.x);
                x[u][1] = __ldcs(at.x + (c + u < p.n_parts ? p.tile : rg));
                advance(at, c + u);
            }
        }
    };
    load(c_begin);
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kJoinUnroll; ++u) top = fmaxf(top, w[u].x);
    Place far = at;
    for (int c = c_begin + kJoinUnroll; c < c_end; ++c) {
        top = fmaxf(top, far.ml->x);
        advance(far, c);
    }
    s_top[run][lane] = top;
    __syncthreads();
    top = fmaxf(fmaxf(s_top[0][lane], s_top[1][lane]), fmaxf(s_top[2][lane], s_top[3][lane]));
    if (top == -INFINITY) top = 0.f;
    float l = 0.f;
    float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int c = c_begin; c < c_end; c += kJoinUnroll) {
        if (c > c_begin) load(c);
#pragma unroll
        for (int u = 0; u < kJoinUnroll; ++u) {
            if (c + u >= c_end) break;
            const float f = ex2_approx((w[u].x - top) * kScaleLog2);
            l = fmaf(w[u].y, f, l);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                o[i].x = fmaf(x[u][i].x, f, o[i].x);
                o[i].y = fmaf(x[u][i].y, f, o[i].y);
                o[i].z = fmaf(x[u][i].z, f, o[i].z);
                o[i].w = fmaf(x[u][i].w, f, o[i].w);
            }
        }
    }
    if (run != 0) {
        s_o[run][0][lane] = o[0];
        s_o[run][1][lane] = o[1];
    }
    s_l[run][lane] = l;
    __syncthreads();
    if (run != 0 || v >= p.n_vec) return;
    l = s_l[0][lane];
    uint4 y = make_uint4(0u, 0u, 0u, 0u);       // idle
#pragma unroll
    for (int r = 1; r < kJoinRuns; ++r) {
        l += s_l[r][lane];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 t = s_o[r][i][lane];
            o[i] = make_float4(o[i].x + t.x, o[i].y + t.y, o[i].z + t.z, o[i].w + t.w);
        }
    }
    if (n > 0) {
        auto pair = [&](float e0, float e1) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__fdiv_rn(e0, l), __fdiv_rn(e1, l));
            return *reinterpret_cast<const uint32_t *>(&h);
        };
        y = make_uint4(pair(o[0].x, o[0].y), pair(o[0].z, o[0].w), pair(o[1].x, o[1].y), pair(o[1].z, o[1].w));
    }
    const int row = idx_div(v, a.group);
    *reinterpret_cast<uint4 *>(a.out + (size_t)row * a.ldo + (size_t)(j * a.group + v - row * a.group) * kHeadDim + 4 * quad) = y;
}

// cuTensorMapEncodeTiled, or null where the driver has none.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool there = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                               cudaSuccess &&
                           q == cudaDriverEntryPointSuccess;
        return there ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

bool encode(CUtensorMap *m, const void *base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
            const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle, const char **why) {
    const cuuint32_t ones[3] = {1, 1, 1};
    const auto fn = tensor_map_encoder();
    if (!fn) {
        *why = "cuTensorMapEncodeTiled is unavailable";
        return false;
    }
    if (fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, ones,
           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
        *why = "cuTensorMapEncodeTiled rejected the layout";
        return false;
    }
    return true;
}

// Innermost first: an entry's 128 elements, entries, (sequence, head).  The cache
// is stored with its 16-byte chunks already permuted by position, as the
// 128-byte swizzle wants them in shared memory, so the copy permutes nothing.
bool encode_cache(CUtensorMap *m, const void *base, int rows, int max_len, int outer, const char **why) {
    return encode(m, base, {cuuint64_t(kHeadDim), cuuint64_t(rows), cuuint64_t(outer)},
                  {cuuint64_t(kHeadDim) * 2, cuuint64_t(max_len) * kHeadDim * 2}, {64, kTile, 1},
                  CU_TENSOR_MAP_SWIZZLE_NONE, why);
}

// Innermost first: a head's 128 elements, heads, rows.
bool encode_queries(CUtensorMap *m, const AttnBatchArgs &a, const char **why) {
    return encode(m, a.q, {cuuint64_t(kHeadDim), cuuint64_t(a.own.n_kv) * a.group, cuuint64_t(a.own.n_seq) * a.R},
                  {cuuint64_t(kHeadDim) * 2, cuuint64_t(a.ldq) * 2},
                  {64, cuuint32_t(a.group), cuuint32_t(kTile / a.group)}, CU_TENSOR_MAP_SWIZZLE_128B, why);
}

}  // namespace

// Workspace: the status block, whose byte 128 is the item counter, then the lane
// GEMM's split-K counters, not used here, then the parts' results.  No operator
// has scratch in the status block, so the counter is zero whatever a workspace
// was used for before, and a GEMM that uses it next finds its counters as it left them.
constexpr size_t kCounterAt = 128, kResultsAt = 256 + kCounterBytes;

size_t attn_batch_bytes(const KvBatch &own, int prefix_len, int group, int R) {
    const Plan p = plan_of(own, prefix_len, group, R);
    return kResultsAt + size_t(p.slots) * (kHeadDim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_attn_batch(const AttnBatchArgs &a, cudaStream_t s, const char **why) {
    static std::atomic<bool> opted_in[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !opted_in[dev]) {
        e = cudaFuncSetAttribute(attn_batch_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(kSmemBytes<false>));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(attn_batch_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     int(kSmemBytes<true>));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) opted_in[dev] = true;
    }
    KernelArgs k{};
    k.a = a;
    k.p = plan_of(a.own, a.prefix_len, a.group, a.R);
    char *base = static_cast<char *>(a.ws);
    k.next = reinterpret_cast<unsigned *>(base + kCounterAt);
    k.opart = reinterpret_cast<float *>(base + kResultsAt);
    k.ml = reinterpret_cast<float2 *>(base + kResultsAt + size_t(k.p.slots) * kHeadDim * sizeof(float));
    const bool e4m3 = a.own.format == kKvE4m3;
    if (!encode_queries(&k.map[4], a, why)) return cudaErrorInvalidValue;
    if (!e4m3) {
        const KvBatch &pre = a.prefix_len > 0 ? a.prefix : a.own;
        const int pre_rows = a.prefix_len > 0 ? a.prefix_len : a.own.max_len;
        if (!encode_cache(&k.map[0], pre.k, pre_rows, pre.max_len, pre.n_kv, why) ||
            !encode_cache(&k.map[1], pre.v, pre_rows, pre.max_len, pre.n_kv, why) ||
            !encode_cache(&k.map[2], a.own.k, a.own.max_len, a.own.max_len, a.own.n_seq * a.own.n_kv, why) ||
            !encode_cache(&k.map[3], a.own.v, a.own.max_len, a.own.max_len, a.own.n_seq * a.own.n_kv, why))
            return cudaErrorInvalidValue;
    }
    const long long items = (long long)a.own.n_kv * ((long long)k.p.n_parts * k.p.pairs +
                                                     (long long)a.own.n_seq * k.p.own_parts_max);
    const int sms = device_sm_count();
    const dim3 grid(unsigned(items < sms ? items : sms));
    e = e4m3 ? launch_pdl(attn_batch_kernel<true>, grid, dim3(Form<true>::threads), kSmemBytes<true>, s, k)
             : launch_pdl(attn_batch_kernel<false>, grid, dim3(Form<false>::threads), kSmemBytes<false>, s, k);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_batch_join_kernel, dim3((k.p.n_vec + 31) / 32, a.own.n_kv, 16), dim3(kJoinThreads), 0, s, a, k.p,
                      (const float *)k.opart, (const float2 *)k.ml, k.next);
}

}  // namespace tfk
