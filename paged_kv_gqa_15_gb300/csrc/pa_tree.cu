// pa_tree.cu -- attention of drafted token trees over the paged cache, on the Blackwell
// tensor cores.
//
// What it computes: sequence b's cache ends in its T drafted nodes (the last T of its L
// tokens); row i of the tree and query head h attend to the C = L - T context tokens
// (under a sliding window, those from C + n_i - window on, n_i the nodes the row sees) and
// to the nodes named by the row's bit mask; softmax(sm_scale q . k) weighted sum of v.
//
// The key axis is read once for all T rows and all query heads of a kv head, so up to about
// 280 rows (T x group) the call is bound by streaming K and V (4 flops a row and element of
// 4 bytes against 286 flops a byte of the GPU).  The design follows from that:
//  * Rows are packed for the MMA's M = 128: row r of a tile is node r / g, query head r % g of
//    one kv head, loaded by one TMA box (64 columns, g heads, 128 / g nodes).  A tree with
//    more rows takes several row tiles, worked on side by side where that pays (TreeShares).
//  * The work is a line of key tiles: for every (sequence, kv head, row tile) its 64-key
//    tiles, one after another.  CTA c of n takes an equal share of that line (one tile more at
//    most), whatever the lengths: no list is sorted and no counter claimed.  Where runs are short
//    against a share, the cuts move to the nearest run boundaries (a share is then up to a run
//    longer than another); where row tiles go side by side (TreeShares), CTAs whose sequence has
//    no such row tile are idle.  A share is a run of segments; a segment that holds all tiles of its
//    (sequence, kv head, row tile) writes the output, the others (at most two per CTA: its
//    first and its last) write fp32 partial rows that a second kernel joins in a fixed order,
//    so results do not depend on timing.
//  * 6 warps: TMA producer (K, V pages through two rings, block tables a tile ahead), MMA
//    issuer (S_j = Q K_j^T into TMEM, O += P_{j-1} V_{j-1} with P from TMEM), four softmax
//    warps with a query row per thread.  Two CTAs share an SM at head_dim <= 128, so one
//    streams and multiplies while the other's softmax runs.  Softmax warps whose rows are all
//    empty skip the arithmetic: a tree of 8 nodes and 4 heads costs one warp's.
//  * Only tiles that reach into the drafted nodes, the edge of a window or a bad page are
//    masked: there each row's visible keys of a tile are one 64-bit word, put together from
//    the context's run of keys and the row's mask words.
//  * P is 0 for a key that a row does not see, but 0 x NaN would poison the row all the same,
//    and rows see different nodes.  So in those tiles the softmax warps also clean V: rows
//    past the sequence are zeroed, and non-finite elements of partly seen rows are zeroed and
//    noted, to be added in the epilogue to the rows that do see them.
//  * 8-bit caches (FP8): K and V tiles go to the 8-bit tensor cores as they are, and MMAs with
//    the same B operand add up the terms of the other.  q is split into two E4M3 rows, q s =
//    hi + lo with s a power of two that puts the row's largest |q s| in [128, 256).  hi takes the
//    four leading bits of bf16's eight and lo the others, so the pair is exact where |q s| >= 2^-2;
//    below, E4M3's smallest step leaves up to 2^-10: 2^-17 of the row's largest |q| (a channel
//    2^13 times the others leaves them a few bits).  P is split into three E5M2 terms: an f16 value's upper byte
//    is an E5M2 value, so each term is a mask and a subtraction and four of them one byte
//    permutation.  Three terms hold at least 9 bits, rounded (2^-9 of P, mostly better), over f16's
//    range.
//    P as E4M3 pairs has one product less and was 8 % faster in an earlier build (154 us against 167
//    for 32 sequences of 1k-8k, 64-node trees), but E4M3 reaches from 448 to 2^-9
//    only: weights far under one large maximum lost their bits, and they can be most of the sum.
//    Two more warps turning V into f16 left too little shared memory for tiles on their way: 261 us.
//  * Every mbarrier wait is bounded.
// Measured: 8 sequences of 32k-131k tokens, 24 nodes, 32 / 8 heads, bf16: 338 us for 2236 MB, 97 % of
// the measured copy rate; 16 of 512-4096 tokens, 16 nodes: 36 us for 130 MB, start and join
// included; 32 of 1k-8k over an FP8 cache, 64 nodes: 160 us for 75 GFLOP, bound by the latency of
// the softmax of 256 rows (tensor pipe 36 % busy, issue slots 37 %) between five MMA terms.
#include <algorithm>
#include <atomic>

#include <cuda.h>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRows = 128;          // rows of a tile (MMA M)
constexpr int kKeys = 64;           // keys of a tile
constexpr int kPages = kKeys / kBlockSize;
constexpr int kTreeThreads = 192;
constexpr int kMaxCtas = 304;       // two per SM of 152
constexpr int kMaxSeqs = 960;       // sequences per launch (their prefix is in shared memory)

// A cut run costs a partial tile's way out and back and a second kernel's work: more than this many
// tiles where the GPU is full (32 sequences of 500 tokens, 8 tiles a run, 128 rows: 39.6 us cut
// evenly, 26.0 in whole runs; at 4000 tokens the two are level), and no more where it is not (3
// sequences of 232-618 tokens at head_dim 256: 15 us cut, 25 in whole runs).
constexpr int kCutTiles = 6;

// Runs cut into this many pieces or more on average are joined by eight warps a row (4 runs of 680
// tiles, 76 pieces each: 39 -> 29 us; 28 runs, 11 pieces: 20 -> 23 us).
constexpr int kManyPieces = 12;

constexpr uint32_t pow2_columns(uint32_t x) {
    uint32_t v = 32;
    while (v < x) v <<= 1;
    return v;
}

template <int HD, bool FP8>
struct TreeCfg {
    static constexpr int ROWB = HD * (FP8 ? 1 : 2) < 128 ? HD * (FP8 ? 1 : 2) : 128;  // bytes of a chunk's row
    static constexpr int CH = HD * (FP8 ? 1 : 2) / ROWB;          // column chunks of a row
    static constexpr int COLS = HD / CH;                          // elements of a chunk's row
    static constexpr uint32_t ATOM = 8 * ROWB;                    // swizzle atom (8 rows)
    static constexpr uint32_t Q_CHUNK = kRows * ROWB;
    static constexpr uint32_t Q_BYTES = (FP8 ? 2 : 1) * CH * Q_CHUNK;   // FP8: hi rows, then lo rows
    static constexpr uint32_t KV_CHUNK = kKeys * ROWB;
    static constexpr uint32_t KV_BYTES = CH * KV_CHUNK;
    // Ring stages: as many tiles as two CTAs' (one at head_dim 256) shared memory holds
    static constexpr int STAGES = HD == 256 ? (FP8 ? 4 : 2) : (HD == 128 ? (FP8 ? 4 : 2) : (FP8 ? 8 : 4));
    // With two stages, K stage t % 2 is free once S_t is done, which s_full[t % 2] says: one commit
    // less per tile (the next phase of s_full needs a K tile that the producer has not sent).
    static constexpr bool K_BY_S = STAGES == 2;
    static constexpr uint32_t OFF_K = Q_BYTES;
    static constexpr uint32_t OFF_V = OFF_K + STAGES * KV_BYTES;
    static constexpr uint32_t OFF_PREF = OFF_V + STAGES * KV_BYTES;    // int64 [kMaxSeqs + 1]
    static constexpr uint32_t OFF_RUN = OFF_PREF + (kMaxSeqs + 1) * 8; // int [kMaxSeqs + 1]
    static constexpr uint32_t OFF_BAR = OFF_RUN + (kMaxSeqs + 2) * 4;
    static constexpr uint32_t SMEM_USED = OFF_BAR + 1280;
    static constexpr int CTAS_PER_SM = HD == 256 ? 1 : 2;
    static constexpr uint32_t SMEM = SMEM_USED + 1024;           // + realignment of the base
    static constexpr uint32_t TM_O = 2 * kKeys;                  // TMEM: S / P twice, then O
    static constexpr uint32_t TMEM_COLS = pow2_columns(2 * kKeys + HD);
    static_assert(CTAS_PER_SM * TMEM_COLS <= 512, "TMEM");
    static_assert(CTAS_PER_SM * (SMEM + 2048) <= 228 * 1024, "shared memory");
};

// A run of tiles that was cut, as the CTA of its second piece notes it (pieces = 0: none).
struct TreeCut {
    int pieces;        // shares it lies in, from the one before on
    int rows, head;    // rows of its row tile, kernel head group
    int node0;         // first row of q and out
    int stride;        // CTAs from one of its shares to the next
};

struct TreeLaunch {
    CUtensorMap tm_q, tm_k, tm_v;   // q only for bf16 caches (FP8 splits q itself)
    TreeParams p;
    float *part_o;                  // [2 grid][rows][HD], unnormalised
    float2 *part_ml;                // [2 grid][rows]: maximum (log2 units) and sum
    TreeCut *cuts;                  // [grid]
    int group, kv_rep, heads;       // query heads per kernel group, groups per kv head, groups
    int nodes;                      // nodes of a row tile (its rows: nodes * group)
    int slot_rows;                  // rows of a partial slot
    int max_ctas;                   // bound of the grid
    bool lists;                     // one query per sequence over page lists (launch_page_lists)
    bool whole;                     // no run is to be cut (there is no room for partial rows)
    int ctas;                       // of the grid
};

// Slot of the partial rows of a run that starts or ends in CTA cta's share (`starts`: it starts
// there).  Trees: two slots a CTA, for its first and its last run.  Page lists, whose workspace is
// that of the split decode: the pieces are numbered along the line, where each next one lies in the
// next share, the next run or both, so share + run is theirs alone (a run is its sequence's row
// and head; there is one row tile).
template <bool LISTS>
__device__ __forceinline__ int piece_slot(const TreeLaunch &a, int cta, bool starts, int row0, int head) {
    return LISTS ? cta + row0 * a.heads + head : 2 * cta + (starts ? 1 : 0);
}

// Sequence b's drafted rows and lengths; T = 0 (and the device status set when `flag`) if
// they make no sense, a length past the table among them: its nodes are then not in the table.
// (A page list that claims more tokens than it has pages ends with its pages, as in the split decode.)
struct TreeSeq {
    int row0, T, L;
};

template <bool LISTS>
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int b, bool flag) {
    TreeSeq s;
    s.row0 = LISTS ? b : p.qo_indptr[b];
    const int row1 = LISTS ? b + 1 : p.qo_indptr[b + 1];
    s.L = max(p.seq_lens[b], 0);
    const int cap = p.max_blocks * kBlockSize;
    bool bad = s.L > cap;
    s.L = min(s.L, cap);
    s.T = 0;
    if (LISTS)
        s.T = 1;
    else if (!bad && s.row0 >= 0 && row1 >= s.row0 && row1 <= p.total_rows && row1 - s.row0 <= p.max_tree_len &&
        row1 - s.row0 <= s.L)
        s.T = row1 - s.row0;
    else
        bad = true;
    if (flag && bad) atomicOr(p.status, kStatusBounds);
    return s;
}

// First key any row could see (a row that sees no node sees from C - window on).
__device__ __forceinline__ int tree_first_key(const TreeSeq &s, int window) {
    return window > 0 ? max(0, s.L - s.T - window) : 0;
}

// Key tiles of one (sequence, kv head, row tile); one that masks everything for an empty page list.
__device__ __forceinline__ int tree_tiles(const TreeSeq &s, int window) {
    // (a table may hold up to 2^31 - 16 tokens: L + 63 would not fit)
    return s.T > 0 ? (s.L - 1) / kKeys + 1 - tree_first_key(s, window) / kKeys : 0;
}

// Row tiles that go together are worked on by as many CTAs at once (see TreeShares); with fewer
// rows than that in some sequences, some of those CTAs are idle there: no more than a quarter of
// the work may be.  bf16 only: over 8-bit caches wide trees are bound by their products and not by
// reading (32 sequences of 1k-8k, 64-node trees: 174 us side by side, 167 one after another;
// bf16 140 against 155, and 549 against 675 for 8 of 32k-131k).
constexpr int kMostTogether = 8;

// pref[b] = tiles of the line before sequence b, run[b] the tiles of its runs, run[n] those of
// the longest, run[n + 1] the row tiles that go together; all threads of the CTA call it, with
// pref[0], run[n] and run[n + 1] cleared.
template <bool FP8, bool LISTS>
__device__ __forceinline__ void tree_prefix(const TreeLaunch &a, int64_t *pref, int *run, bool flag) {
    const TreeParams &p = a.p;
    const int n = p.num_seqs;
    int most_tiles = 0, most_rows = 0;
    for (int b = threadIdx.x; b < n; b += kTreeThreads) {
        const TreeSeq s = tree_seq<LISTS>(p, b, flag);
        const int tiles = tree_tiles(s, p.window), row_tiles = (s.T + a.nodes - 1) / a.nodes;
        run[b] = tiles;
        pref[b + 1] = static_cast<int64_t>(tiles) * row_tiles * a.heads;
        most_tiles = max(most_tiles, tiles);
        most_rows = max(most_rows, row_tiles);
    }
    most_tiles = __reduce_max_sync(kAll, most_tiles);
    most_rows = __reduce_max_sync(kAll, most_rows);
    if ((threadIdx.x & 31) == 0) {
        atomicMax(&run[n], most_tiles);
        atomicMax(&run[n + 1], most_rows);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int together = run[n + 1];
        bool pair = !FP8 && together > 1 && together <= kMostTogether;
        if (pair) {
            long long apart = 0, once = 0;   // tiles with row tiles one after another, and side by side
            for (int b = lane; b < n; b += 32) {
                apart += pref[b + 1];
                once += static_cast<long long>(run[b]) * a.heads;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                apart += __shfl_xor_sync(kAll, apart, o);
                once += __shfl_xor_sync(kAll, once, o);
            }
            pair = once * together * 3 <= apart * 4;
        }
        __syncwarp();
        if (pair)
            for (int b = lane; b < n; b += 32) pref[b + 1] = static_cast<int64_t>(run[b]) * a.heads;
        else if (lane == 0)
            run[n + 1] = 1;
        __syncwarp();
        long long carry = 0;
        for (int base = 1; base <= p.num_seqs; base += 32) {
            const int i = base + lane;
            long long v = i <= p.num_seqs ? pref[i] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(kAll, v, o);
                if (lane >= o) v += u;
            }
            if (i <= p.num_seqs) pref[i] = v + carry;
            carry += __shfl_sync(kAll, v, 31);
        }
    }
    __syncthreads();
}

// How the line of tiles is cut into shares: evenly, or at the run boundaries nearest to the
// even cuts, which needs no joining.  Where trees take several row tiles, that many CTAs take
// one share together, a row tile each, and so read the same keys at about the same time: the
// second comes from L2.  (One after another in the line, the row tiles of 8 sequences of 32k-131k
// tokens with 64-node trees read every key from HBM twice: 675 us.)
struct TreeShares {
    const int64_t *pref;   // [n + 1] tiles before sequence b
    const int *run;        // [n] tiles of each of sequence b's runs
    int64_t total, even;   // total = even * shares + more
    int n, shares, more;
    bool whole;

    // x / d and x % d, in 32 bits where they do (64-bit division is a hundred instructions)
    static __device__ __forceinline__ int quotient(int64_t x, int d) {
        return x <= INT32_MAX ? static_cast<int>(x) / d : static_cast<int>(x / d);
    }
    static __device__ __forceinline__ int remainder(int64_t x, int d) {
        return x <= INT32_MAX ? static_cast<int>(x) % d : static_cast<int>(x % d);
    }
    // the largest b with pref[b] <= u, by a whole warp: every stride-th prefix, then those between
    __device__ __forceinline__ int sequence(int64_t u) const {
        const int lane = threadIdx.x & 31, stride = (n + 31) >> 5;
        const int lo = (__popc(__ballot_sync(kAll, lane * stride < n && pref[lane * stride] <= u)) - 1) * stride;
        if (stride == 1) return lo;
        return lo + __popc(__ballot_sync(kAll, lane < stride && lo + lane < n && pref[lo + lane] <= u)) - 1;
    }
    // the share tile u lies in, of an even cut
    __device__ __forceinline__ int share_of(int64_t u) const {
        const int64_t longer = (even + 1) * more;   // tiles of the shares that are one longer
        return u < longer ? quotient(u, static_cast<int>(even) + 1)
                          : more + quotient(u - longer, static_cast<int>(even));
    }
    __device__ __forceinline__ int64_t begin(int c) const {
        if (c >= shares) return total;
        const int64_t u = even * c + min(c, more);
        if (!whole || u <= 0) return u;
        const int b = sequence(u);
        const int r = remainder(u - pref[b], run[b]);
        return 2 * r >= run[b] ? u - r + run[b] : u - r;
    }
};

// One run of a share's tiles within one (sequence, kv head, row tile).
struct TreeSegment {
    int b, head, node0, n_nodes;   // kernel head group; first node of the row tile, nodes in it
    int row0, T, L;
    int j0, n;                     // first key tile (of the sequence) and tiles; n = -1: no more
    int page_lo;                   // first page that any row sees (window)
    int slot;                      // partial slot, or -1: all tiles are here
};

struct TreeQueue {
    TreeSegment seg[4];
    uint32_t bad_nodes[16];        // partly seen rows with non-finite values (see the cleaning of V)
    uint32_t bad_pages[16];        // ring by tile: pages whose ids are out of range
    float row_factor[kRows];       // FP8: the power of two that q's rows are scaled by
};

__device__ __forceinline__ TreeSegment read_again(const TreeSegment &s) {
    const volatile TreeSegment &v = s;
    TreeSegment r;
    r.b = v.b, r.head = v.head, r.node0 = v.node0, r.n_nodes = v.n_nodes;
    r.row0 = v.row0, r.T = v.T, r.L = v.L;
    r.j0 = v.j0, r.n = v.n, r.page_lo = v.page_lo, r.slot = v.slot;
    return r;
}
static_assert(48 * 8 + sizeof(TreeQueue) <= 1280, "queue fits behind the barriers");

__device__ __forceinline__ uint64_t ones(int n) { return n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1); }

// Word w of a row's mask, without bits past the tree.
__device__ __forceinline__ uint64_t mask_word(const uint64_t *mask, int w, int T) {
    return w * 64 < T ? mask[w] & ones(T - w * 64) : 0ull;
}

// The block-table row of sequence b for pool kv head kvh.
template <bool LISTS>
__device__ __forceinline__ const int32_t *tree_table_row(const TreeParams &p, int b, int kvh) {
    return p.block_tables + (LISTS ? static_cast<int64_t>(b) * p.num_kv_heads + kvh : b) * p.max_blocks;
}

__device__ __forceinline__ int mask_count(const uint64_t *mask, int T) {
    int n = 0;
    for (int w = 0; w * 64 < T; ++w) n += __popcll(mask_word(mask, w, T));
    return n;
}

// The 64 mask bits from bit `at` (which may be negative) on; word0 is the mask's first word.
__device__ __forceinline__ uint64_t mask_bits_at(const uint64_t *mask, uint64_t word0, int at, int T) {
    if (at <= -64 || at >= T) return 0;
    if (at < 0) return word0 << -at;
    const uint64_t lo = (at < 64 ? word0 : mask_word(mask, at >> 6, T)) >> (at & 63);
    return at & 63 ? lo | mask_word(mask, (at >> 6) + 1, T) << (64 - (at & 63)) : lo;
}

// Swizzled byte offset of 16-byte unit c of row r in a chunk whose rows have ROWB bytes.
template <int ROWB>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    return ROWB == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Zeroes the non-finite elements of a 16-byte unit; whether there were any.
template <bool FP8>
__device__ __forceinline__ bool drop_non_finite(uint4 &v) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t keep = 0xffffffffu;
        if constexpr (FP8) {   // E4M3 has NaN alone: 0x7f, 0xff
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if ((w[i] >> 8 * e & 0x7f) == 0x7f) keep &= ~(0xffu << 8 * e);
        } else {
            if ((w[i] & 0x7f80u) == 0x7f80u) keep &= 0xffff0000u;
            if ((w[i] & 0x7f800000u) == 0x7f800000u) keep &= 0x0000ffffu;
        }
        any |= keep != 0xffffffffu;
        w[i] &= keep;
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
    return any;
}

// Four P values (0 to 2^15) as E5M2 codes of three terms that add up to them: by way of f16,
// whose upper byte is the value cut to E5M2; what is cut off goes to the next term, exactly.  The
// last term is rounded (cut, it left P up to 2^-8 too small and the outputs, whose sum of weights
// is not cut, 2^-10 on average): half a step up for two keys, a hair less for the next two, so that
// what lies half-way between does not all go one way.
__device__ __forceinline__ void split_e5m2x4(float x0, float x1, float x2, float x3, uint32_t (&t)[3]) {
    uint32_t a, b;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(a) : "f"(x1), "f"(x0));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(x3), "f"(x2));
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (i == 2) a += 0x00800080u, b += 0x007f007fu;
        t[i] = __byte_perm(a, b, 0x7531);   // the upper bytes
        if (i == 2) break;
        const uint32_t ta = a & 0xff00ff00u, tb = b & 0xff00ff00u;
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(a) : "r"(ta));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(b) : "r"(tb));
    }
}

// The largest magnitude of eight bf16 values.
__device__ __forceinline__ float largest(const uint4 &raw) {
    float f[8], most = 0.f;
    unpack_bf16x8(raw, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(f[e]));
    return most;
}

// The power of two s with most * s in [128, 256); an infinite row becomes NaN, as its scores are.
__device__ __forceinline__ float row_factor(float most) {
    const int ex = static_cast<int>(__float_as_uint(most) >> 23 & 0xff);
    if (ex == 255) return NAN;
    return ex > 0 ? __uint_as_float(static_cast<uint32_t>(min(max(127 + 7 + 127 - ex, 1), 254)) << 23) : 1.f;
}

// 16 channels of q (unit c of its row) times s as E4M3 pairs, into Q's hi and lo rows.
template <typename C>
__device__ __forceinline__ void store_pair(uint8_t *q, int row, int c, const uint4 &a, const uint4 &b, float s) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        float f[8];
        unpack_bf16x8(v ? b : a, f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t h[2], l[2];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const float x = f[4 * e + 2 * d] * s, y = f[4 * e + 2 * d + 1] * s;
                h[d] = float2_to_e4m3x2(x, y);
                const float2 back = e4m3x2_to_float2(h[d]);
                l[d] = float2_to_e4m3x2(x - back.x, y - back.y);
            }
            hi[2 * v + e] = h[0] | h[1] << 16;
            lo[2 * v + e] = l[0] | l[1] << 16;
        }
    }
    constexpr int UNITS = C::ROWB / 16;
    uint8_t *dst = q + (c / UNITS) * C::Q_CHUNK + swizzled<C::ROWB>(row, c % UNITS);
    *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(dst + C::CH * C::Q_CHUNK) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// LISTS: one query per sequence over page lists (launch_page_lists), as a tree of one node, the
// list's last key, which sees itself.
template <int HD, bool FP8, bool LISTS>
__global__ void __launch_bounds__(kTreeThreads, TreeCfg<HD, FP8>::CTAS_PER_SM)
    tree_kernel(const __grid_constant__ TreeLaunch a) {
    using C = TreeCfg<HD, FP8>;
    const TreeParams &p = a.p;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    int64_t *pref = reinterpret_cast<int64_t *>(smem + C::OFF_PREF);
    int *run = reinterpret_cast<int *>(smem + C::OFF_RUN);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    // Tiles are numbered g over all segments of the CTA: ring stage g % STAGES, S buffer g % 2.
    uint64_t *q_full = bars + 0;     // FP8: one arrival per softmax warp
    uint64_t *q_empty = bars + 1;    // the segment's last S is done (commit)
    uint64_t *o_free = bars + 2;     // the epilogue has read O (one arrival per softmax warp)
    uint64_t *drain = bars + 3;
    uint64_t *s_full = bars + 4;     // [2] S_g is done (commit)
    uint64_t *p_full = bars + 6;     // [2] P_g is in TMEM, V_g is clean (one arrival per softmax warp)
    uint64_t *k_full = bars + 8;     // [STAGES <= 8]
    uint64_t *k_empty = bars + 16;   // [STAGES] (commit)
    uint64_t *v_full = bars + 24;
    uint64_t *v_empty = bars + 32;   // P_g V_g is done (commit)
    uint64_t *seg_full = bars + 40;  // [4]
    uint64_t *seg_empty = bars + 44; // [4]: the MMA thread and 4 softmax warps
    TreeQueue *queue = reinterpret_cast<TreeQueue *>(bars + 48);
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // rows of Q past the row tile stay zero, so that their scores are numbers
    for (uint32_t i = threadIdx.x; i < C::Q_BYTES / 16; i += kTreeThreads)
        reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x < 16) queue->bad_nodes[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        pref[0] = 0;
        run[p.num_seqs] = run[p.num_seqs + 1] = 0;
        mbar_init(q_full, FP8 ? 4 : 1);
        mbar_init(q_empty, 1);
        mbar_init(o_free, 4);
        mbar_init(drain, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
        }
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&seg_full[s], 1);
            mbar_init(&seg_empty[s], 5);
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&a.tm_k);
        prefetch_tensormap(&a.tm_v);
        if (!FP8) prefetch_tensormap(&a.tm_q);
    }
    fence_proxy_async_smem();   // the zeroed rows are read by the tensor core
    if (warp == 1) {
        tmem_alloc(&tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp >= 2) {   // the first reads after the wait, into L2 beforehand
        const unsigned t = blockIdx.x * 128 + threadIdx.x - 64, nt = gridDim.x * 128;
        prefetch_decode_inputs(p.seq_lens, p.block_tables, p.q, p.num_seqs, LISTS ? p.num_kv_heads : 1, p.max_blocks,
                               static_cast<size_t>(p.total_rows) * p.num_q_heads * HD * 2, threadIdx.x - 64, 128);
        if constexpr (!LISTS) {
            prefetch_l2_lines(p.qo_indptr, (static_cast<size_t>(p.num_seqs) + 1) * 4, t, nt);
            prefetch_l2_lines(p.tree_mask, static_cast<size_t>(p.total_rows) * p.mask_words * 8, t, nt);
        }
    }
    // launched as a programmatic dependent: nothing before this point depends on global memory
    __syncthreads();   // what tree_prefix adds to is cleared
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tree_prefix<FP8, LISTS>(a, pref, run, blockIdx.x == 0);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    const int together = run[p.num_seqs + 1];
    const int share = static_cast<int>(blockIdx.x) / together, member = static_cast<int>(blockIdx.x) % together;
    TreeShares line{pref, run, pref[p.num_seqs], 0, p.num_seqs, static_cast<int>(gridDim.x) / together, 0, false};
    if (line.total < line.shares) line.shares = max(1, static_cast<int>(line.total));
    line.even = line.total <= INT32_MAX ? static_cast<int>(line.total) / line.shares : line.total / line.shares;
    line.more = static_cast<int>(line.total - line.even * line.shares);
    {
        // Shares of whole runs hold at most one run when there are no more runs than shares, else
        // an even share and a run.
        const int64_t longest = run[p.num_seqs];
        const int64_t most = line.even < longest ? longest : line.even + longest;
        line.whole = (LISTS && a.whole) || most <= line.even + kCutTiles;
    }
    const int64_t u_begin = line.begin(share);
    const int64_t u_end = line.begin(share + 1);

    if (warp == 0) {
        // ------------------------------- TMA producer -------------------------------
        uint32_t g = 0, n_seg = 0;
        uint32_t n_k = 0, n_v = 0, n_q = 0;   // copies issued (for the drain on an abort)
        int stop = 0;
        int64_t u = u_begin;
        int64_t run_begin = -1, run_end = -1; // of a run that began in a share before
        // Publishes the next segment of the share (or the end) and returns it.
        auto next_segment = [&]() -> TreeSegment {
            const int slot = n_seg & 3;
            TreeSegment s = {};
            s.n = -1;
            while (u < u_end) {
                const int lo = line.sequence(u);
                const TreeSeq q = tree_seq<LISTS>(p, lo, false);
                const int tiles = run[lo];
                const int row_tiles = together > 1 ? 1 : (q.T + a.nodes - 1) / a.nodes;
                const int64_t rel = u - pref[lo];
                const int item = TreeShares::quotient(rel, tiles);
                const int j = static_cast<int>(rel - static_cast<int64_t>(item) * tiles);
                const int n = static_cast<int>(min(static_cast<int64_t>(tiles - j), u_end - u));
                const int node0 = (together > 1 ? member : item % row_tiles) * a.nodes;
                if (node0 >= q.T) {   // the sequence has no such row tile
                    u += n;
                    continue;
                }
                s.b = lo;
                s.head = item / row_tiles;
                s.node0 = node0;
                s.n_nodes = min(a.nodes, q.T - s.node0);
                s.row0 = q.row0;
                s.T = q.T;
                s.L = q.L;
                s.n = n;
                s.j0 = tree_first_key(q, p.window) / kKeys + j;
                s.slot = s.n == tiles ? -1 : piece_slot<LISTS>(a, static_cast<int>(blockIdx.x), j == 0, s.row0, s.head);
                if (j > 0) {   // only in the share's first segment
                    run_begin = u - j;
                    run_end = run_begin + tiles;
                }
                if (p.window > 0) {   // pages before the first key a row does see are not looked up
                    int least = 1 << 30;
                    for (int i = lane; i < q.T; i += 32)
                        least = min(least, mask_count(p.tree_mask + static_cast<int64_t>(q.row0 + i) * p.mask_words, q.T));
#pragma unroll
                    for (int o = 16; o; o >>= 1) least = min(least, __shfl_xor_sync(kAll, least, o));
                    s.page_lo = max(0, min(q.L - q.T, q.L - q.T + least - p.window)) / kBlockSize;
                }
                u += n;
                break;
            }
            if (lane == 0) {
                if (!mbar_wait(&seg_empty[slot], ((n_seg >> 2) & 1) ^ 1u, p.status, abort_flag)) {
                    stop = 1;
                } else {
                    queue->seg[slot] = s;
                    mbar_arrive(&seg_full[slot]);
                }
            }
            ++n_seg;
            stop = __shfl_sync(kAll, stop, 0);
            if (stop) s.n = -1;
            return s;
        };
        // Block-table entry of page `lane` of key tile j; -2 for pages no row sees.
        auto page_raw = [&](const TreeSegment &s, int j) -> int {
            const int i = j * kPages + lane;
            if (lane >= kPages || i * kBlockSize >= s.L || i < s.page_lo) return -2;
            return tree_table_row<LISTS>(p, s.b, s.head / a.kv_rep)[i];
        };
        const uint64_t policy = l2_policy_evict_first();
        TreeSegment w = next_segment();
        const TreeCut run_cut = {2, w.n_nodes * a.group, w.head, w.row0 + w.node0, together};
        bool noted = false;
        // Where the share before holds the run's first piece, this one has it joined; written
        // behind the first loads, since nothing here waits for it.
        auto note_cut = [&]() {
            if (noted) return;
            noted = true;
            TreeCut cut = {};
            if (run_begin >= 0 && run_begin >= line.begin(share - 1)) {
                cut = run_cut;
                cut.pieces = line.share_of(run_end - 1) - share + 2;
            }
            if (lane == 0 && !(LISTS && a.whole)) a.cuts[blockIdx.x] = cut;
        };
        while (!stop && w.n >= 0) {
            const int kvh = w.head / a.kv_rep;
            if (!FP8) {
                if (lane == 0) {
                    if (n_q > 0 && !mbar_wait(q_empty, (n_q - 1) & 1, p.status, abort_flag)) stop = 1;
                    else mbar_arrive_expect_tx(q_full, C::CH * a.nodes * a.group * C::ROWB);
                }
                stop = __shfl_sync(kAll, stop, 0);
                if (stop) break;
                if (lane < C::CH)
                    tma_load_3d(smem + lane * C::Q_CHUNK, &a.tm_q, lane * C::COLS, w.head * a.group,
                                w.row0 + w.node0, q_full);
                ++n_q;
            }
            // Loads tile j's keys (kv = 0) or values (kv = 1); t is its number over all segments.
            auto load = [&](int kv, uint32_t t, int page) {
                const int s = t % C::STAGES;
                const uint32_t ph = ((t / C::STAGES) & 1) ^ 1u;
                uint64_t *full = kv ? &v_full[s] : &k_full[s];
                if (lane == 0) {
                    uint64_t *empty = kv ? &v_empty[s] : (C::K_BY_S ? &s_full[s] : &k_empty[s]);
                    if (!mbar_wait(empty, ph, p.status, abort_flag)) stop = 1;
                    else mbar_arrive_expect_tx(full, C::KV_BYTES);
                }
                stop = __shfl_sync(kAll, stop, 0);
                if (stop) return;
                ++(kv ? n_v : n_k);
                const int pg = __shfl_sync(kAll, page, lane / C::CH);
                if (lane < kPages * C::CH)   // lane l: chunk l % CH of page l / CH
                    tma_load_4d_hint(smem + (kv ? C::OFF_V : C::OFF_K) + s * C::KV_BYTES +
                                         (lane % C::CH) * C::KV_CHUNK + (lane / C::CH) * kBlockSize * C::ROWB,
                                     kv ? &a.tm_v : &a.tm_k, (lane % C::CH) * C::COLS, 0, kvh, pg, full, policy);
            };
            // Ids out of range become an out-of-range box, which reads zeros; their keys are
            // masked through bad_pages, which the softmax reads after S_t: the entry of tile t
            // is written again with tile t + 16, long after (K runs at most STAGES + 1 ahead).
            auto page_fix = [&](int raw, uint32_t t) -> int {
                const bool bad = raw != -2 && (raw < 0 || raw >= p.num_blocks);
                const unsigned which = __ballot_sync(kAll, bad);
                if (lane == 0) {
                    queue->bad_pages[t & 15] = which;
                    if (which) atomicOr(p.status, kStatusBounds);
                }
                return raw == -2 || bad ? static_cast<int>(p.num_blocks) : raw;
            };
            int page = page_fix(page_raw(w, w.j0), g);
            int raw = w.n > 1 ? page_raw(w, w.j0 + 1) : -2;
            load(0, g, page);
            TreeSegment next = w;
            for (int j = 0; j < w.n && !stop; ++j) {
                if (j == 1) note_cut();
                int page_next = 0;
                if (j + 1 < w.n) {
                    page_next = page_fix(raw, g + j + 1);
                    if (j + 2 < w.n) raw = page_raw(w, w.j0 + j + 2);
                    load(0, g + j + 1, page_next);
                }
                if (!stop) load(1, g + j, page);
                page = page_next;
                // the segment behind is looked up once this one's first tiles are on their way
                if (j == 0 && !stop) next = next_segment();
            }
            g += w.n;
            w = next;
        }
        note_cut();
        // never leave the CTA with copies still landing in its shared memory
        if (lane == 0 && (stop || *abort_flag)) {
            auto settle = [&](uint64_t *full, int ns, uint32_t n) {
                for (uint32_t k = n > static_cast<uint32_t>(ns) ? n - ns : 0; k < n; ++k) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(&full[k % ns], (k / ns) & 1u))
                        if (global_timer_ns() - t0 > kWaitLimitNs) break;
                }
            };
            settle(q_full, 1, n_q);
            settle(k_full, C::STAGES, n_k);
            settle(v_full, C::STAGES, n_v);
        }
    } else if (warp == 1) {
        // -------------------------------- MMA issuer --------------------------------
        if (lane == 0) {
            constexpr uint32_t idesc_s = FP8 ? idesc_f32(kRows, kKeys, 0, 0, false, false)
                                             : idesc_bf16_f32(kRows, kKeys, false, false);
            // P: three terms of E5M2 (format 1)
            constexpr uint32_t idesc_o = FP8 ? idesc_f32(kRows, HD, 1, 0, false, true)
                                             : idesc_bf16_f32(kRows, HD, false, true);
            constexpr int KB = 32;                         // bytes of K per MMA
            constexpr int PER_CHUNK = C::ROWB / KB;        // MMAs per chunk of a row
            constexpr int PV_ROWS = FP8 ? 32 : 16;         // keys per P.V MMA
            constexpr uint32_t sbo = C::ATOM;
            const uint64_t q_desc = smem_desc_sw<C::ROWB>(smem_addr(smem), 16, sbo);
            const uint64_t k_desc = smem_desc_sw<C::ROWB>(smem_addr(smem + C::OFF_K), 16, sbo);
            const uint64_t v_desc = smem_desc_sw<C::ROWB>(smem_addr(smem + C::OFF_V), C::KV_CHUNK, sbo);
            uint32_t g = 0;
            bool ok = true;
            auto issue_pv = [&](uint32_t t, bool first, uint32_t segment) {
                if (!ok) return;
                const int s = t % C::STAGES;
                if (first && segment > 0)   // the segment before has read O
                    ok = mbar_wait(o_free, (segment - 1) & 1, p.status, abort_flag);
                ok = ok && mbar_wait(&p_full[t & 1], (t >> 1) & 1, p.status, abort_flag) &&
                     mbar_wait(&v_full[s], (t / C::STAGES) & 1, p.status, abort_flag);
                if (!ok) return;
                tc_fence_after_sync();
                const uint64_t vd = v_desc + ((s * C::KV_BYTES) >> 4);
                const uint32_t pt = tmem + (t & 1) * kKeys;
#pragma unroll
                for (int part = 0; part < (FP8 ? 3 : 1); ++part)
#pragma unroll
                    for (int kk = 0; kk < kKeys / PV_ROWS; ++kk) {
                        const uint64_t d = vd + ((kk * PV_ROWS * C::ROWB) >> 4);
                        const uint32_t acc = !first || kk > 0 || part > 0 ? 1u : 0u;
                        if constexpr (FP8) mma_f8_ts(tmem + C::TM_O, pt + part * 16 + kk * 8, d, idesc_o, acc);
                        else mma_bf16_ts(tmem + C::TM_O, pt + kk * 8, d, idesc_o, acc);
                    }
                tc_commit(&v_empty[s]);
            };
            for (uint32_t k = 0; ok; ++k) {
                const int slot = k & 3;
                ok = mbar_wait(&seg_full[slot], (k >> 2) & 1, p.status, abort_flag);
                if (!ok) break;
                const int n = queue->seg[slot].n;
                mbar_arrive(&seg_empty[slot]);
                if (n < 0) break;
                ok = mbar_wait(q_full, k & 1, p.status, abort_flag);
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t t = g + j;
                    const int s = t % C::STAGES;
                    ok = mbar_wait(&k_full[s], (t / C::STAGES) & 1, p.status, abort_flag);
                    if (!ok) break;
                    tc_fence_after_sync();
                    // S buffer t % 2 held P_{t-2}, whose P.V was issued by this thread before
                    const uint64_t kd = k_desc + ((s * C::KV_BYTES) >> 4);
#pragma unroll
                    for (int part = 0; part < (FP8 ? 2 : 1); ++part)
#pragma unroll
                        for (int kk = 0; kk < C::CH * PER_CHUNK; ++kk) {
                            const uint32_t c = kk / PER_CHUNK, in = (kk % PER_CHUNK) * KB;
                            const uint64_t qd = q_desc + (((part * C::CH + c) * C::Q_CHUNK + in) >> 4);
                            const uint64_t d = kd + ((c * C::KV_CHUNK + in) >> 4);
                            const uint32_t acc = kk > 0 || part > 0 ? 1u : 0u;
                            if constexpr (FP8) mma_f8_ss(tmem + (t & 1) * kKeys, qd, d, idesc_s, acc);
                            else mma_bf16_ss(tmem + (t & 1) * kKeys, qd, d, idesc_s, acc);
                        }
                    tc_commit(&s_full[t & 1]);
                    if (!C::K_BY_S) tc_commit(&k_empty[s]);
                    if (j == n - 1) tc_commit(q_empty);
                    if (j > 0) issue_pv(t - 1, j == 1, k);
                }
                issue_pv(g + n - 1, n == 1, k);
                g += n;
            }
            tc_commit(drain);   // never release TMEM or shared memory with MMAs in flight
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(drain, 0)) {
                if (global_timer_ns() - t0 > kWaitLimitNs) {
                    atomicOr(p.status, kStatusTimeout);
                    break;
                }
            }
        }
        __syncwarp();
    } else {
        // ----------------------------- softmax and epilogue -----------------------------
        const int quad = warp & 3;                 // TMEM lane quadrant of this warp
        const int row = quad * 32 + lane;          // row of the tile
        const int tid = threadIdx.x - 64;          // 0 .. 127 over the softmax warps
        const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
        // A row's maximum moves only when it grows by more than 2^8: O is then rescaled rarely,
        // and bf16 holds any P.  FP8: 2^(8 + 7) is within f16 and E5M2, whose smallest step is 2^-16.
        constexpr float lag = 8.f;
        constexpr float lift = FP8 ? 7.f : 0.f;    // P is 2^(x - m + lift)
        uint32_t g = 0;
        bool ok = true;
        for (uint32_t k = 0;; ++k) {
            const int slot = k & 3;
            ok = mbar_wait(&seg_full[slot], (k >> 2) & 1, p.status, abort_flag);
            // the four warps leave the loop at the same barrier, after a wait that ran out too
            if (named_barrier_or(1, 128, !ok)) break;
            const TreeSegment w = queue->seg[slot];
            if (w.n < 0) break;
            const int rows = w.n_nodes * a.group;
            const bool busy = quad * 32 < rows;    // this warp has rows
            const bool mine = row < rows;
            const int ctx = w.L - w.T;
            const uint64_t *mask = LISTS ? nullptr : p.tree_mask + static_cast<int64_t>(w.row0 + w.node0 + (mine ? row / a.group : 0)) * p.mask_words;
            // read now: the tile that needs it would wait for it
            const uint64_t word0 = !mine ? 0ull : LISTS ? 1ull : mask_word(mask, 0, w.T);
            int low = 0;                           // first context token this row sees
            if (p.window > 0) low = max(0, min(ctx, ctx + mask_count(mask, w.T) - p.window));
            const int seen_by_all = p.window > 0 ? max(0, min(ctx, ctx + w.T - p.window)) : 0;
            const int first_key = p.window > 0 ? max(0, ctx - p.window) : 0;
            float scale = p.scale_log2;
            if constexpr (FP8) {
                // q's rows as E4M3 pairs, once the segment before has finished with Q
                if (k > 0) ok = mbar_wait(q_empty, (k - 1) & 1, p.status, abort_flag);
                ok = !__any_sync(kAll, !ok);
                // four threads a row, a quarter of its channels each, 32 rows at a time
#pragma unroll 1
                for (int r0 = 0; r0 < rows; r0 += 32) {
                    const int r = r0 + (tid >> 2), part = tid & 3;
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        static_cast<const __nv_bfloat16 *>(p.q) +
                        (static_cast<int64_t>(w.row0 + w.node0 + r / a.group) * p.num_q_heads + w.head * a.group +
                         r % a.group) * HD) + part * (HD / 32);
                    uint4 held[HD / 32];
#pragma unroll
                    for (int c = 0; c < HD / 32; ++c) held[c] = r < rows ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                    float most = 0.f;
#pragma unroll
                    for (int c = 0; c < HD / 32; ++c) most = fmaxf(most, largest(held[c]));
                    most = fmaxf(most, __shfl_xor_sync(kAll, most, 1));
                    most = fmaxf(most, __shfl_xor_sync(kAll, most, 2));
                    const float s = row_factor(most);
#pragma unroll
                    for (int c = 0; c < HD / 64; ++c)
                        store_pair<C>(smem, r, part * (HD / 64) + c, held[2 * c], held[2 * c + 1], s);
                    if (part == 0) queue->row_factor[r] = s;
                }
                named_barrier(1, 128);
                // above zero: -inf times it stays so
                if (mine) scale = fmaxf(p.scale_log2 * p.k_scale / queue->row_factor[row], 0x1p-126f);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            float m = -INFINITY, l = 0.f;          // running maximum (log2 units) and sum
            for (int j = 0; j < w.n && ok; ++j) {
                const uint32_t t = g + j;
                const uint32_t s_col = (t & 1) * kKeys;
                ok = mbar_wait(&s_full[t & 1], (t >> 1) & 1, p.status, abort_flag);
                if (__any_sync(kAll, !ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const int base = (w.j0 + j) * kKeys;
                const uint32_t bad_pages = *static_cast<volatile uint32_t *>(&queue->bad_pages[t & 15]);
                const bool edge = base + (kKeys - 1) >= ctx || base < seen_by_all || bad_pages;
                if (__builtin_expect(edge && (base + (kKeys - 1) >= ctx || base < seen_by_all), 0)) {
                    // Clean V: rows that no row sees are zeroed (past the sequence, before the
                    // window), partly seen ones lose and note what is not finite.
                    const int s = t % C::STAGES;
                    ok = mbar_wait(&v_full[s], (t / C::STAGES) & 1, p.status, abort_flag);
                    if (__any_sync(kAll, !ok)) {
                        ok = false;
                        break;
                    }
                    uint8_t *vt = smem + C::OFF_V + s * C::KV_BYTES;
                    for (int i = tid; i < static_cast<int>(C::KV_BYTES / 16); i += 128) {
                        const int key = base + i % static_cast<int>(C::KV_CHUNK / 16) / (C::ROWB / 16);
                        if (key >= seen_by_all && key < ctx) continue;
                        uint4 *unit = reinterpret_cast<uint4 *>(vt) + i;
                        if (key >= w.L || key < first_key) {
                            *unit = make_uint4(0u, 0u, 0u, 0u);
                        } else {
                            uint4 v = *unit;
                            if (drop_non_finite<FP8>(v)) {
                                *unit = v;
                                const int at = key >= ctx ? key - ctx : 256 + key - first_key;
                                atomicOr(&queue->bad_nodes[at >> 5], 1u << (at & 31));
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                if (busy) {
                    uint32_t sr[kKeys];
                    tmem_load_64(tmem + t_lane + s_col, sr);
                    if (__builtin_expect(edge, 0)) {
                        uint64_t see = 0;
                        if (mine) {
                            see = (ones(ctx - base) & ~ones(low - base)) | mask_bits_at(mask, word0, base - ctx, w.T);
#pragma unroll
                            for (int e = 0; e < kPages; ++e)
                                if (bad_pages >> e & 1) see &= ~(0xffffull << e * kBlockSize);
                        }
                        const uint32_t see_lo = static_cast<uint32_t>(see), see_hi = static_cast<uint32_t>(see >> 32);
#pragma unroll
                        for (int c = 0; c < kKeys; ++c)
                            if (!((c < 32 ? see_lo : see_hi) >> (c & 31) & 1)) sr[c] = __float_as_uint(-INFINITY);
                    }
                    float mx[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx[e] = fmaxf(__uint_as_float(sr[e]), __uint_as_float(sr[8 + e]));
#pragma unroll
                    for (int c = 16; c < kKeys; c += 16)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            mx[e] = fmax3(mx[e], __uint_as_float(sr[c + e]), __uint_as_float(sr[c + 8 + e]));
                    const float top = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                    const float m_new = fmaxf(m, top * scale);
                    const bool grow = m_new > m + lag;
                    const float corr = !grow ? 1.f : (m == -INFINITY ? 0.f : fast_exp2(m - m_new));
                    if (j > 0 && __any_sync(kAll, grow)) {
                        // O holds the tiles before: wait for the last P.V, then rescale in TMEM
                        const uint32_t b = t - 1;
                        ok = mbar_wait(&v_empty[b % C::STAGES], (b / C::STAGES) & 1, p.status, abort_flag);
                        if (__any_sync(kAll, !ok)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
#pragma unroll
                        for (int c = 0; c < HD / 32; ++c) {
                            uint32_t o[32];
                            tmem_load_32(tmem + t_lane + C::TM_O + c * 32, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                            tmem_store_32(tmem + t_lane + C::TM_O + c * 32, o);
                        }
                        tmem_store_wait();
                    }
                    if (grow) {
                        l *= corr;
                        m = m_new;
                    }
                    // P = 2^(s scale - m + lift).  The sum takes the fp32 values, P goes to the MMA as bf16,
                    // the type of the tile it multiplies: nearest, so off by 2^-9 of a weight on average
                    // and either way (outputs 2.3e-3 from 64 bits in relative norm, 1.7e-3 of it their own
                    // rounding to bf16).
                    const float sub = m == -INFINITY ? 0.f : m - lift;
                    constexpr int P_WORDS = FP8 ? 48 : 32;
                    uint32_t pk[P_WORDS];
                    float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                     make_float2(0.f, 0.f)};
                    const float2 sc2 = make_float2(scale, scale), nm2 = make_float2(-sub, -sub);
#pragma unroll
                    for (int c = 0; c < kKeys / 2; c += 2) {
                        float2 e[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[2 * (c + i)]),
                                                                    __uint_as_float(sr[2 * (c + i) + 1])), sc2, nm2);
                            e[i] = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                            sum[(c + i) & 3] = __fadd2_rn(sum[(c + i) & 3], e[i]);
                        }
                        if constexpr (FP8) {
                            uint32_t t3[3];
                            split_e5m2x4(e[0].x, e[0].y, e[1].x, e[1].y, t3);
#pragma unroll
                            for (int i = 0; i < 3; ++i) pk[i * 16 + c / 2] = t3[i];
                        } else {
                            pk[c] = pack_bf16x2(e[0].x, e[0].y);
                            pk[c + 1] = pack_bf16x2(e[1].x, e[1].y);
                        }
                    }
                    const float2 s01 = __fadd2_rn(sum[0], sum[1]), s23 = __fadd2_rn(sum[2], sum[3]);
                    const float2 st = __fadd2_rn(s01, s23);
                    l += st.x + st.y;
                    tmem_store_32(tmem + t_lane + s_col, *reinterpret_cast<uint32_t (*)[32]>(&pk[0]));
                    if constexpr (FP8)
                        tmem_store_16(tmem + t_lane + s_col + 32, *reinterpret_cast<uint32_t (*)[16]>(&pk[32]));
                    tmem_store_wait();
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t & 1]);
            }
            g += w.n;
            // O is final once the segment's last P.V is done
            ok = ok && mbar_wait(&v_empty[(g - 1) % C::STAGES], ((g - 1) / C::STAGES) & 1, p.status, abort_flag);
            if (named_barrier_or(1, 128, !ok)) break;
            tc_fence_after_sync();
            // read again: what only the epilogue needs is not held in registers through the tiles
            const TreeSegment e = read_again(queue->seg[slot]);
            const int node = e.node0 + (mine ? row / a.group : 0);
            const int head = e.head * a.group + (mine ? row % a.group : 0);
            const bool whole = e.slot < 0;
            const float inv = l > 0.f ? p.v_scale / l : (l == 0.f ? 0.f : l);   // a NaN sum stays one
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) +
                                 (static_cast<int64_t>(e.row0 + node) * p.num_q_heads + head) * HD;
            float *part = a.part_o + (static_cast<int64_t>(max(e.slot, 0)) * a.slot_rows + row) * HD;
            if (busy) {
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t o[32];
                    tmem_load_32(tmem + t_lane + C::TM_O + c * 32, o);
                    if (mine && whole) {
                        uint32_t v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            v[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<uint4 *>(out + c * 32)[e] =
                                make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    } else if (mine) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)   // whole sectors
                            st_global_32B(part + c * 32 + e, o[e], o[e + 1], o[e + 2], o[e + 3], o[e + 4], o[e + 5],
                                          o[e + 6], o[e + 7]);
                    }
                    __syncwarp();
                }
                if (mine && !whole) a.part_ml[static_cast<int64_t>(e.slot) * a.slot_rows + row] = make_float2(m, l);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            // What the clean-up took out of V goes to the rows that see it (rare: a non-finite
            // value in a drafted node's row).  P.V of every tile is done, so every warp has
            // noted what it found.
            uint32_t found = 0;
            if (lane < 16) found = *static_cast<volatile uint32_t *>(&queue->bad_nodes[lane]);
            if (__any_sync(kAll, found != 0)) {
                if (mine) {
                    for (int at = 0; at < 512; ++at) {
                        if (!(*static_cast<volatile uint32_t *>(&queue->bad_nodes[at >> 5]) >> (at & 31) & 1)) continue;
                        const int key = at < 256 ? ctx + at : first_key + at - 256;
                        const bool see = at >= 256 ? key >= low
                                         : LISTS   ? at == 0
                                                   : (mask_word(mask, at >> 6, e.T) >> (at & 63) & 1);
                        if (!see) continue;
                        const int page = tree_table_row<LISTS>(p, e.b, e.head / a.kv_rep)[key / kBlockSize];
                        const int64_t off = page * p.s_block + (e.head / a.kv_rep) * p.s_head +
                                            (key % kBlockSize) * p.s_token;
                        for (int d = 0; d < HD; ++d) {
                            const float v = FP8 ? e4m3x2_to_float2(static_cast<const uint8_t *>(p.v_cache)[off + d]).x
                                                : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.v_cache)[off + d]);
                            if (isfinite(v)) continue;
                            if (whole) out[d] = __float2bfloat16_rn(__bfloat162float(out[d]) + v);
                            else part[d] += v;
                        }
                    }
                }
                __syncwarp();
            }
            // the notes are the segment's own: all four warps have read them before they are cleared
            const bool clear = named_barrier_or(1, 128, found != 0);
            if (clear) {
                if (tid < 16) queue->bad_nodes[tid] = 0;
                named_barrier(1, 128);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[slot]);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// One warp's sum over `count` partial rows, slot(0), slot(1), ...: the running maximum and sum, and
// acc, whose lane holds channels lane, lane + 32, ...  The maxima and sums of up to 32 pieces are read
// at once, one per lane, and the partial rows four at a time: a few memory round trips, not one per
// piece.
template <int HD, typename Slot>
__device__ __forceinline__ void join_pieces(const TreeLaunch &a, Slot slot, int count, float &m, float &l,
                                            float (&acc)[HD / 32]) {
    constexpr int D = HD / 32, U = 4;
    const int lane = threadIdx.x & 31;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int d = 0; d < D; ++d) acc[d] = 0.f;
    for (int base = 0; base < count; base += 32) {
        const int n = min(32, count - base);
        const float2 ml = lane < n ? a.part_ml[slot(base + lane)] : make_float2(-INFINITY, 0.f);
        float top = fmaxf(m, ml.x);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        const float f = m == -INFINITY ? 0.f : exp2f(m - top);
        const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : ml.y) : exp2f(ml.x - top);   // keeps a NaN
        float sum = w * ml.y;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        l = l * f + sum;
#pragma unroll
        for (int d = 0; d < D; ++d) acc[d] *= f;
        m = top;
        for (int i = 0; i < n; i += U) {
            float o[U][D];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float *src = a.part_o + slot(base + min(i + u, n - 1)) * HD;
#pragma unroll
                for (int d = 0; d < D; ++d) o[u][d] = src[d * 32 + lane];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float wu = __shfl_sync(kAll, w, min(i + u, n - 1));
                if (i + u < n && wu != 0.f) {
#pragma unroll
                    for (int d = 0; d < D; ++d) acc[d] = fmaf(o[u][d], wu, acc[d]);
                }
            }
        }
    }
}

// Partial row of piece i of a run whose second piece is CTA `cta`'s: piece 0 is the last run of the
// share before, the others are the first runs of theirs.
__device__ __forceinline__ int64_t piece_row(const TreeLaunch &a, const TreeCut &cut, int cta, int row, int i) {
    const int c = cta + (i - 1) * cut.stride;
    const int slot = a.lists ? piece_slot<true>(a, c, i == 0, cut.node0, cut.head)
                             : piece_slot<false>(a, c, i == 0, cut.node0, cut.head);
    return static_cast<int64_t>(slot) * a.slot_rows + row;
}

template <int HD>
__device__ __forceinline__ __nv_bfloat16 *joined_row(const TreeLaunch &a, const TreeCut &cut, int row) {
    const int64_t node = cut.node0 + row / a.group;
    const int h = cut.head * a.group + row % a.group;
    return static_cast<__nv_bfloat16 *>(a.p.out) + (node * a.p.num_q_heads + h) * HD;
}

__device__ __forceinline__ float joined_scale(const TreeLaunch &a, float l) {
    return l > 0.f ? a.p.v_scale / l : (l == 0.f ? 0.f : l);
}

// Joins the partial rows of every (sequence, kernel head group, row tile) that was cut: one
// warp per row, the shares' partials in a fixed order, so the result does not depend on
// timing.  Grid: x = CTA, y = eight rows; the CTA that had a cut run's second piece stands for
// it.  Bound by its round trips to memory and its launch: 6 us for the cut runs of 304 shares of 32
// rows, 12 for 128 rows (the partial rows, up to 40 MB, mostly come from L2).
template <int HD>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ TreeLaunch a) {
    constexpr int D = HD / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cta = static_cast<int>(blockIdx.x) + 1;
    const TreeCut cut = a.cuts[cta];
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (cut.pieces == 0 || row >= cut.rows) return;
    float m, l, acc[D];
    join_pieces<HD>(a, [&](int i) { return piece_row(a, cut, cta, row, i); }, cut.pieces, m, l, acc);
    __nv_bfloat16 *out = joined_row<HD>(a, cut, row);
    const float inv = joined_scale(a, l);
#pragma unroll
    for (int d = 0; d < D; ++d) out[d * 32 + lane] = __float2bfloat16_rn(acc[d] * inv);
}

// The same where few long runs are cut into many pieces each: eight warps share a row, every eighth
// piece each, and add up in shared memory in the order of the warps.  Grid: x = eight CTAs, y = row.
// (One sequence of 43545 tokens, 4 kv heads, 76 pieces a run: a warp per row took 18 us of the call.)
template <int HD>
__global__ void __launch_bounds__(256) tree_join_long_kernel(const __grid_constant__ TreeLaunch a) {
    constexpr int D = HD / 32;
    __shared__ float part[8][HD];
    __shared__ float2 part_ml[8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y;
    const int cta0 = static_cast<int>(blockIdx.x) * 8 + 1;
    const bool cuts_run = lane < 8 && cta0 + lane < a.ctas && a.cuts[cta0 + lane].pieces > 0;
    for (unsigned which = __ballot_sync(kAll, cuts_run); which; which &= which - 1) {   // the same in every warp
        const int cta = cta0 + __ffs(which) - 1;
        const TreeCut cut = a.cuts[cta];
        if (row >= cut.rows) continue;
        float m, l, acc[D];
        join_pieces<HD>(a, [&](int i) { return piece_row(a, cut, cta, row, warp + 8 * i); },
                        (cut.pieces - warp + 7) / 8, m, l, acc);
        __syncthreads();   // the run before has been read
#pragma unroll
        for (int d = 0; d < D; ++d) part[warp][d * 32 + lane] = acc[d];
        if (lane == 0) part_ml[warp] = make_float2(m, l);
        __syncthreads();
        float top = -INFINITY, sum = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) top = fmaxf(top, part_ml[w].x);
        for (int c = threadIdx.x; c < HD; c += 256) {
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const float2 ml = part_ml[w];
                const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : ml.y) : exp2f(ml.x - top);
                sum += f * ml.y;
                if (f != 0.f) o = fmaf(part[w][c], f, o);
            }
            joined_row<HD>(a, cut, row)[c] = __float2bfloat16_rn(o * joined_scale(a, sum));
        }
    }
}

// ---- host side ------------------------------------------------------------------------------

// The kernel's groups of query heads: the whole group of a kv head, or its largest divisor
// that fits the row tile.
int tree_group(int num_q_heads, int num_kv_heads) {
    const int G = num_q_heads / num_kv_heads;
    int g = G < kRows ? G : kRows;
    while (G % g) --g;
    return g;
}

int tree_nodes(int group, int max_tree_len) {
    const int n = kRows / group;
    return n < max_tree_len ? n : max_tree_len;
}

template <int HD, bool FP8, bool LISTS>
cudaError_t launch_tree(TreeLaunch &a, cudaStream_t stream) {
    using C = TreeCfg<HD, FP8>;
    const TreeParams &p = a.p;
    if (!FP8) {
        const cuuint64_t dims[3] = {HD, static_cast<cuuint64_t>(p.num_q_heads),
                                    static_cast<cuuint64_t>(p.total_rows)};
        const cuuint64_t str[2] = {HD * 2, static_cast<cuuint64_t>(p.num_q_heads) * HD * 2};
        const cuuint32_t box[3] = {C::COLS, static_cast<cuuint32_t>(a.group), static_cast<cuuint32_t>(a.nodes)};
        if (!encode_tensor_map_bf16(&a.tm_q, p.q, 3, dims, str, box)) return cudaErrorInvalidValue;
    }
    {
        constexpr int E = FP8 ? 1 : 2;
        const cuuint64_t dims[4] = {HD, kBlockSize, static_cast<cuuint64_t>(p.num_kv_heads),
                                    static_cast<cuuint64_t>(p.num_blocks)};
        const cuuint64_t str[3] = {static_cast<cuuint64_t>(p.s_token) * E, static_cast<cuuint64_t>(p.s_head) * E,
                                   static_cast<cuuint64_t>(p.s_block) * E};
        const cuuint32_t box[4] = {C::COLS, kBlockSize, 1, 1};
        auto encode = FP8 ? encode_tensor_map_u8 : encode_tensor_map_bf16;
        if (!encode(&a.tm_k, p.k_cache, 4, dims, str, box) || !encode(&a.tm_v, p.v_cache, 4, dims, str, box))
            return cudaErrorInvalidValue;
    }
    auto kern = tree_kernel<HD, FP8, LISTS>;
    static std::atomic<int> configured{-1};   // last device whose attributes are set
    static std::atomic<int> sm_count{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (configured.load() != dev) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        sm_count = n;
        configured = dev;
    }
    const int sms = sm_count.load();
    // no more CTAs than the longest possible line has tiles
    const int row_tiles = (p.max_tree_len + a.nodes - 1) / a.nodes;
    const int64_t line = static_cast<int64_t>(p.num_seqs) * a.heads * row_tiles *
                         ((static_cast<int64_t>(p.max_blocks) * kBlockSize + kKeys - 1) / kKeys);
    int grid = std::min(sms * C::CTAS_PER_SM, a.max_ctas);
    if (line < grid) grid = static_cast<int>(line);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    a.ctas = grid;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess) return e;
    // Runs of at most kCutTiles are never cut (TreeShares::whole), and one share cuts nothing.
    int64_t longest = (static_cast<int64_t>(p.max_blocks) * kBlockSize + kKeys - 1) / kKeys;
    if (p.window > 0)
        longest = std::min(longest, (static_cast<int64_t>(p.window) + p.max_tree_len + kKeys - 1) / kKeys + 1);
    if (grid == 1 || longest <= kCutTiles || a.whole) return cudaSuccess;
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    if (grid >= static_cast<int64_t>(kManyPieces) * p.num_seqs * a.heads * row_tiles) {
        cfg.gridDim = dim3(static_cast<unsigned>((grid + 6) / 8), static_cast<unsigned>(a.slot_rows));
        return cudaLaunchKernelEx(&cfg, tree_join_long_kernel<HD>, a);
    }
    cfg.gridDim = dim3(static_cast<unsigned>(grid - 1), static_cast<unsigned>((a.slot_rows + 7) / 8));
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<HD>, a);
}

}  // namespace

namespace {

TreeLaunch tree_launch(const TreeParams &p, size_t slots, int head_dim) {
    TreeLaunch a = {};
    a.p = p;
    a.group = tree_group(p.num_q_heads, p.num_kv_heads);
    a.kv_rep = p.num_q_heads / p.num_kv_heads / a.group;
    a.heads = p.num_q_heads / a.group;
    a.nodes = tree_nodes(a.group, p.max_tree_len);
    a.slot_rows = a.nodes * a.group;
    a.max_ctas = kMaxCtas;
    a.part_o = static_cast<float *>(p.workspace);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + slots * a.slot_rows * head_dim);
    a.cuts = reinterpret_cast<TreeCut *>(a.part_ml + slots * a.slot_rows);
    return a;
}

}  // namespace

cudaError_t launch_tree_decode(const TreeParams &p, int head_dim, cudaStream_t stream) {
    TreeLaunch a = tree_launch(p, 2 * kMaxCtas, head_dim);
    // the line's prefix holds kMaxSeqs sequences: more go in several launches, one after another
    for (int at = 0; at < p.num_seqs; at += kMaxSeqs) {
        a.p.num_seqs = std::min(p.num_seqs - at, kMaxSeqs);
        a.p.seq_lens = p.seq_lens + at;
        a.p.qo_indptr = p.qo_indptr + at;
        a.p.block_tables = p.block_tables + static_cast<int64_t>(at) * p.max_blocks;
        cudaError_t e;
        switch (head_dim) {
            case 64: e = p.kv_fp8 ? launch_tree<64, true, false>(a, stream) : launch_tree<64, false, false>(a, stream); break;
            case 128: e = p.kv_fp8 ? launch_tree<128, true, false>(a, stream) : launch_tree<128, false, false>(a, stream); break;
            case 256: e = p.kv_fp8 ? launch_tree<256, true, false>(a, stream) : launch_tree<256, false, false>(a, stream); break;
            default: return cudaErrorNotSupported;
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// A page list is a tree of one node, the list's last key, whose other keys are its context.
// The split decode has no tensor-core kernel for head_dim 256, nor at head_dim 64 for groups above 8
// (over FP8 for any), and walks a list once per sub-group of query heads that it has a kernel for, a
// CTA for every 32 pages.  The tree kernel walks it once, but a list is a chain of tiles to it: about
// 20 us (35 at head_dim 256) for lists of more than 32 pages, down to half of that for short ones,
// however few there are.  So it takes the calls whose CTAs the split decode would need more than a
// wave or two of, half as many where lists are short.
// Measured, split decode / this, us (sequences x kv heads x pages of a list):
//   head_dim 256, group 3: 1 x 8 x 128 14 / 29, 4 x 8 x 64 24 / 34, 8 x 8 x 64 34 / 35, 16 x 8 x 64 62 / 36,
//     8 x 8 x 8 12 / 13, 32 x 8 x 8 25 / 19; group 4: 22 / 29, 22 / 35, 24 / 35, 41 / 35, 13 / 13, 23 / 19;
//     7: 24 / 29, 33 / 34, 61 / 35, 116 / 36, 15 / 13, 45 / 19; 8: 56 / 28, 56 / 34, 58 / 35, 111 / 35, 27 / 13, 51 / 19
//     (FP8 group 4: 21 / 27, 21 / 28, 22 / 29, 39 / 29, 12 / 11, 20 / 20; 8: 74 / 27, 74 / 28, 78 / 29, 151 / 29, 31 / 12, 62 / 20)
//   head_dim 64, group 9: 11 / 20, 14 / 22, 18 / 22, 30 / 23, 10 / 10, 20 / 10;
//     11: 18 / 20, 26 / 22, 42 / 22, 78 / 23, 12 / 10, 32 / 10; 16: 12 / 19, 12 / 22, 17 / 22, 28 / 23, 9 / 10, 20 / 10
//     (FP8 group 3: 11 / 24, 11 / 23, 18 / 23, 27 / 24, 7 / 9, 12 / 10; 5: 11 / 23, 18 / 23, 26 / 23, 41 / 24, 9 / 9, 18 / 10;
//     8: 16 / 21, 16 / 23, 16 / 23, 28 / 24, 9 / 9, 15 / 10; 4, on the split decode: 41 / 41 at 32 x 8 x 128)
bool page_lists_on_tree(const DecodeParams &p, int head_dim) {
    const int group = p.num_q_heads / p.num_kv_heads;
    if (head_dim == 256 ? group < 3 : head_dim != 64 || (p.kv_fp8 ? group < 3 || group == 4 : group <= 8)) return false;
    int sub = 0;                                  // the split decode's sub-groups: on the tensor cores ...
    for (int g = 8; head_dim == 64 && !p.kv_fp8 && g >= 3 && !sub; --g)
        if (group % g == 0) sub = g;
    const bool tensor = sub > 0;
    for (int g = 8; !sub; g /= 2)                 // ... or not
        if (group % g == 0) sub = g;
    const int64_t ctas = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads * (group / sub) * ((p.max_blocks + 31) / 32);
    int border = head_dim == 256 ? (sub == 8 ? 0 : sub == 4 ? 160 : 320) : tensor ? 320 : sub == 8 ? 160 : 640;
    if (p.max_blocks <= 32) border /= 2;
    return ctas >= border && p.scale_log2 > 0.f && p.scale_log2 < INFINITY && p.num_blocks < INT32_MAX;
}

cudaError_t launch_page_lists(const DecodeParams &d, int head_dim, void *workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
    TreeParams p = {};
    p.out = d.out;
    p.q = d.q;
    p.k_cache = d.k_cache;
    p.v_cache = d.v_cache;
    p.block_tables = d.block_tables;
    p.seq_lens = d.seq_lens;
    p.workspace = workspace;
    p.num_blocks = d.num_blocks;
    p.s_block = d.s_block;
    p.s_head = d.s_head;
    p.s_token = d.s_token;
    p.max_tree_len = 1;
    p.num_q_heads = d.num_q_heads;
    p.num_kv_heads = d.num_kv_heads;
    p.max_blocks = d.max_blocks;
    p.kv_fp8 = d.kv_fp8;
    p.scale_log2 = d.scale_log2;
    p.k_scale = d.k_scale;
    p.v_scale = d.v_scale;
    p.status = d.status;
    const int group = tree_group(p.num_q_heads, p.num_kv_heads);
    const size_t slot_bytes = static_cast<size_t>(group) * (static_cast<size_t>(head_dim) * 4 + 8);
    const size_t cut_bytes = kMaxCtas * sizeof(TreeCut);
    const size_t slots = workspace_bytes > cut_bytes ? (workspace_bytes - cut_bytes) / slot_bytes : 0;
    for (int at = 0; at < d.num_seqs; at += kMaxSeqs) {
        p.num_seqs = p.total_rows = std::min(d.num_seqs - at, kMaxSeqs);
        p.seq_lens = d.seq_lens + at;
        p.block_tables = d.block_tables + static_cast<int64_t>(at) * d.num_kv_heads * d.max_blocks;
        p.q = static_cast<const __nv_bfloat16 *>(d.q) + static_cast<int64_t>(at) * d.num_q_heads * head_dim;
        p.out = static_cast<__nv_bfloat16 *>(d.out) + static_cast<int64_t>(at) * d.num_q_heads * head_dim;
        TreeLaunch a = tree_launch(p, slots, head_dim);
        a.lists = true;
        // pieces number fewer than shares + runs
        const int64_t runs = static_cast<int64_t>(p.num_seqs) * a.heads;
        const int64_t shares = static_cast<int64_t>(slots) - runs;
        a.whole = shares <= runs;
        if (!a.whole) a.max_ctas = static_cast<int>(std::min<int64_t>(shares, kMaxCtas));
        const cudaError_t e =
            head_dim == 64 ? (p.kv_fp8 ? launch_tree<64, true, true>(a, stream) : launch_tree<64, false, true>(a, stream))
                           : (p.kv_fp8 ? launch_tree<256, true, true>(a, stream) : launch_tree<256, false, true>(a, stream));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace pa

extern "C" size_t pa_tree_decode_workspace_size(int num_seqs, int max_tree_len, int num_q_heads,
                                                int num_kv_heads, int head_dim) {
    if (num_seqs <= 0 || max_tree_len <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        num_q_heads % num_kv_heads)
        return 0;
    const int group = pa::tree_group(num_q_heads, num_kv_heads);
    const size_t rows = static_cast<size_t>(2 * pa::kMaxCtas) * pa::tree_nodes(group, max_tree_len) * group;
    return rows * (static_cast<size_t>(head_dim) * 4 + 8) + pa::kMaxCtas * sizeof(pa::TreeCut);
}

extern "C" int pa_tree_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *block_tables, const int32_t *seq_lens,
                              const int32_t *qo_indptr, const int64_t *tree_mask, int mask_words,
                              int num_seqs, int total_rows, int max_tree_len, int num_q_heads,
                              int num_kv_heads, int head_dim, int block_size,
                              int max_blocks_per_seq, int64_t num_blocks, int64_t stride_block,
                              int64_t stride_head, int64_t stride_token, float sm_scale,
                              int sliding_window, int kv_dtype, float k_scale, float v_scale,
                              void *workspace, size_t workspace_bytes, void *stream) {
    using namespace pa;
    if (num_seqs < 0 || total_rows < 0)
        return api_fail(PA_ERR_INVALID, "num_seqs %d, total_rows %d", num_seqs, total_rows);
    int rc = api_check_heads(head_dim, num_q_heads, num_kv_heads);
    if (rc) return rc;
    rc = api_check_kv_dtype(kv_dtype, k_scale, v_scale);
    if (rc) return rc;
    rc = api_check_pool(head_dim, block_size, num_blocks, num_kv_heads, stride_block, stride_head,
                        stride_token, kv_dtype);
    if (rc) return rc;
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > INT32_MAX / kBlockSize)
        return api_fail(PA_ERR_INVALID, "max_blocks_per_seq %d", max_blocks_per_seq);
    if (num_blocks >= INT32_MAX)
        return api_fail(PA_ERR_UNSUPPORTED, "num_blocks %lld too large", (long long)num_blocks);
    if (max_tree_len < 0) return api_fail(PA_ERR_INVALID, "max_tree_len %d", max_tree_len);
    if (max_tree_len > PA_MAX_TREE_LEN)
        return api_fail(PA_ERR_UNSUPPORTED, "max_tree_len %d > %d", max_tree_len, PA_MAX_TREE_LEN);
    if (mask_words < (max_tree_len + 63) / 64)
        return api_fail(PA_ERR_INVALID, "mask_words %d: %d nodes need %d", mask_words, max_tree_len,
                        (max_tree_len + 63) / 64);
    if (!(sm_scale > 0.f) || sm_scale == INFINITY)
        return api_fail(PA_ERR_INVALID, "sm_scale must be positive and finite");
    if (num_seqs == 0 || total_rows == 0 || max_tree_len == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !qo_indptr || !tree_mask)
        return api_fail(PA_ERR_INVALID, "null pointer argument");
    const void *ptrs[4] = {out, q, k_cache, v_cache};
    for (const void *ptr : ptrs)
        if (reinterpret_cast<uintptr_t>(ptr) & 15u)
            return api_fail(PA_ERR_INVALID, "out, q and the KV pools must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(tree_mask) & 7u)
        return api_fail(PA_ERR_INVALID, "tree_mask must be 8-byte aligned");
    const size_t need = pa_tree_decode_workspace_size(num_seqs, max_tree_len, num_q_heads,
                                                      num_kv_heads, head_dim);
    if (workspace_bytes < need)
        return api_fail(PA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return api_fail(PA_ERR_WORKSPACE, "workspace must be non-null and 256-byte aligned");
    TreeParams p = {};
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.qo_indptr = qo_indptr;
    p.tree_mask = reinterpret_cast<const uint64_t *>(tree_mask);
    p.workspace = workspace;
    p.num_blocks = num_blocks;
    p.s_block = stride_block;
    p.s_head = stride_head;
    p.s_token = stride_token;
    p.mask_words = mask_words;
    p.num_seqs = num_seqs;
    p.total_rows = total_rows;
    p.max_tree_len = max_tree_len;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.window = sliding_window > 0 ? sliding_window : 0;
    p.kv_fp8 = kv_dtype == PA_KV_FP8_E4M3 ? 1 : 0;
    p.k_scale = p.kv_fp8 ? k_scale : 1.f;
    p.v_scale = p.kv_fp8 ? v_scale : 1.f;
    p.scale_log2 = sm_scale * kLog2e;
    rc = api_status_ptr(&p.status);
    if (rc) return rc;
    const cudaError_t e = launch_tree_decode(p, head_dim, static_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidValue)
        return api_fail(PA_ERR_CUDA, "tensor map encoding failed (cuTensorMapEncodeTiled)");
    if (e != cudaSuccess) return api_cuda_fail(e, "tree decode launch");
    return PA_OK;
}
