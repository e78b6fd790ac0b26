// pa_pages.cu -- per-page bounds of the keys, and the pages a decode step selects by them.
//
// Bounds: for a page and kv head, the smallest and largest key value of every channel over
// the page's rows inside the sequence.  For a query head q, sum_d max(q_d min_d, q_d max_d)
// bounds q . k from above for every key of the page, so the pages with the largest bounds
// are the ones that can hold the keys the query attends to.  Summed over a kv head's group
// of query heads the bound is one inner product,
//     score = sum_d P_d max_d + N_d min_d,  P = sum_h max(q_h, 0), N = sum_h min(q_h, 0),
// because max(q min, q max) is q max for q >= 0 and q min for q < 0: the group costs no more
// than one head, and the pass is bound by reading the bounds (2 head_dim elements a page).
//
// Selection is by exact scores.  A score computed in fp32 is off by at most
//     E = (group + 24) 2^-24 S + 2^-140,  S >= sum_d |P_d max_d| + |N_d min_d| of any ranked page
// (P and N are sums of `group` terms of one sign: group - 1 roundings; a product is rounded
// once at most, added in a chain of up to 16, joined over at most 32 lanes in five sums; S
// itself and T +- 2E are rounded: fewer than group + 24 act on any term.  Products below the
// normal numbers lose up to 2^-150 each).  S is taken once for a group of pages, from the
// largest magnitude of every channel.  With T the f-th largest computed score, a page above
// T + 2E is among the f best and one below T - 2E is not; the band between is scored again in
// fp64 and ranked by (score, page).
#include <atomic>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---- bounds ---------------------------------------------------------------------------------

struct BoundsParams {
    uint8_t *bounds;
    const uint8_t *k_cache;
    const int32_t *block_tables, *seq_lens, *first_tokens;
    int64_t num_blocks, b_block, b_head, b_token;   // strides in bytes
    int num_seqs, num_kv_heads, max_blocks, pages;  // pages: at most per sequence
    int *status;
};

// Two 16-bit lanes of min / max that hand a NaN on.
template <bool FP8>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (FP8) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <bool FP8>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (FP8) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<unsigned short>(two)));
    return h2;
}

// Every value is one of the page's own codes, so the conversion back is exact.
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t h2) {
    unsigned short c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h2));
    return c;
}

// A unit is one (sequence, page, kv head), its heads next to each other; a warp takes kUnits of
// them in a row.  Lane u looks unit u up (lengths and page id: two dependent reads, once per
// warp), and the rows of the next unit are on their way while one is compared.  A row is CPR
// chunks of 16 bytes; a load instruction reads 32 / CPR rows.  Bound by streaming K: 104 us for
// 578 MB of keys (8 prompts of 8k-65k tokens) with their 72 MB of bounds, 92 % of the measured copy
// rate; a warp per unit reached 88 %, its 4 KB waiting for the look-up every time.
constexpr int kUnits = 4;

template <int HD, bool FP8>
__global__ void __launch_bounds__(256) bounds_kernel(const __grid_constant__ BoundsParams p) {
    constexpr int ROW = HD * (FP8 ? 1 : 2);
    constexpr int CPR = ROW / 16;
    constexpr int RPL = 32 / CPR;                 // rows per load
    constexpr int LOADS = kBlockSize / RPL;
    constexpr int W = FP8 ? 8 : 4;                // 16-bit pairs a lane holds
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kUnits + lane;
    const int64_t per_seq = static_cast<int64_t>(p.pages) * p.num_kv_heads;
    const int64_t b = unit / per_seq;
    int my_rows = 0, my_id = 0, my_head = 0;
    if (lane < kUnits && b < p.num_seqs) {
        const int rest = static_cast<int>(unit - b * per_seq);
        my_head = rest % p.num_kv_heads;
        int L = max(p.seq_lens[b], 0);
        const int first = p.first_tokens ? min(max(p.first_tokens[b], 0), L) : 0;
        const int cap = p.max_blocks * kBlockSize;
        bool bad = L > cap;
        L = min(L, cap);
        const int page = first / kBlockSize + rest / p.num_kv_heads;
        // a sequence's first unit sees whether its pages go on past the launch's
        bad = bad || (L + kBlockSize - 1) / kBlockSize - first / kBlockSize > p.pages;
        if (bad && rest == 0) atomicOr(p.status, kStatusBounds);
        // (a page past the table could pass 2^31 tokens)
        my_rows = first < L && page < p.max_blocks ? max(0, min(kBlockSize, L - page * kBlockSize)) : 0;
        if (my_rows > 0) {
            my_id = p.block_tables[b * p.max_blocks + page];
            if (my_id < 0 || my_id >= p.num_blocks) {
                atomicOr(p.status, kStatusBounds);
                my_rows = 0;
            }
        }
    }
    __syncwarp();
    const int c = lane % CPR, r0 = lane / CPR;
    auto load = [&](int u, uint4 (&raw)[LOADS]) {
        const int rows = __shfl_sync(kAll, my_rows, u), id = __shfl_sync(kAll, my_id, u);
        const int kh = __shfl_sync(kAll, my_head, u);
        const uint8_t *src = p.k_cache + id * p.b_block + kh * p.b_head + c * 16;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)   // rows past the sequence repeat its last one
            raw[i] = rows > 0 ? *reinterpret_cast<const uint4 *>(src + min(i * RPL + r0, rows - 1) * p.b_token)
                              : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 raw[2][LOADS];
    load(0, raw[0]);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        if (u + 1 < kUnits) load(u + 1, raw[(u + 1) & 1]);
        uint32_t lo[W], hi[W];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const uint4 &v = raw[u & 1][i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const uint32_t x = FP8 ? e4m3x2_to_f16x2(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu) : w[e % 4];
                lo[e] = i ? min2<FP8>(lo[e], x) : x;
                hi[e] = i ? max2<FP8>(hi[e], x) : x;
            }
        }
#pragma unroll
        for (int off = CPR; off < 32; off <<= 1)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                lo[e] = min2<FP8>(lo[e], __shfl_xor_sync(kAll, lo[e], off));
                hi[e] = max2<FP8>(hi[e], __shfl_xor_sync(kAll, hi[e], off));
            }
        const int rows = __shfl_sync(kAll, my_rows, u), id = __shfl_sync(kAll, my_id, u);
        const int kh = __shfl_sync(kAll, my_head, u);
        if (rows > 0 && lane < CPR) {
            uint8_t *dst = p.bounds + (static_cast<int64_t>(id) * p.num_kv_heads + kh) * 2 * ROW + c * 16;
            uint32_t a[4], z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = FP8 ? f16x2_to_e4m3x2(lo[(2 * e) % W]) | f16x2_to_e4m3x2(lo[(2 * e + 1) % W]) << 16 : lo[e];
                z[e] = FP8 ? f16x2_to_e4m3x2(hi[(2 * e) % W]) | f16x2_to_e4m3x2(hi[(2 * e + 1) % W]) << 16 : hi[e];
            }
            *reinterpret_cast<uint4 *>(dst) = make_uint4(a[0], a[1], a[2], a[3]);
            *reinterpret_cast<uint4 *>(dst + ROW) = make_uint4(z[0], z[1], z[2], z[3]);
        }
        __syncwarp();
    }
}

// Launches a kernel as a programmatic dependent of the work before it in the stream: its CTAs may
// start while that finishes, and wait for it before they read anything.
template <typename Kernel, typename Params>
cudaError_t launch_after(Kernel kern, dim3 grid, int threads, const Params &p, cudaStream_t stream,
                         size_t smem = 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int HD>
cudaError_t launch_bounds(const BoundsParams &p, bool fp8, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(p.num_seqs) * p.pages * p.num_kv_heads;
    const dim3 grid(static_cast<unsigned>((units + 8 * kUnits - 1) / (8 * kUnits)));
    return fp8 ? launch_after(bounds_kernel<HD, true>, grid, 256, p, stream)
               : launch_after(bounds_kernel<HD, false>, grid, 256, p, stream);
}

// ---- scores ---------------------------------------------------------------------------------


struct SelectParams {
    int32_t *page_tables, *page_lens;
    const __nv_bfloat16 *q;
    const uint8_t *bounds;
    const int32_t *block_tables, *seq_lens;
    float *score;       // [B][nkv][max_blocks]
    float *span;        // [B][nkv][groups]: largest S of a group's ranked pages (0: it has none)
    double *exact;      // [B][nkv][max_blocks], of the pages that are scored again
    int64_t num_blocks;
    int num_seqs, nq, nkv, max_blocks, group, groups, max_pages, sink, recent;   // group: pages of one S
    int *status;
};

__device__ __forceinline__ int select_len(const SelectParams &p, int b, bool flag) {
    int L = max(p.seq_lens[b], 0);
    if (L > p.max_blocks * kBlockSize) {
        if (flag) atomicOr(p.status, kStatusBounds);
        L = p.max_blocks * kBlockSize;
    }
    return L;
}

// The larger number, or NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest of three magnitudes, or NaN if one is.
__device__ __forceinline__ float most_of(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A channel whose query weight is zero adds nothing, an infinite bound included.
template <typename T>
__device__ __forceinline__ T weighed(T w, T x) {
    return w == T(0) ? T(0) : w * x;
}

// 16 bytes of global memory to shared memory, past L1, without a register in between.
__device__ __forceinline__ void cp_async_16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Element d of a bounds row as a float.
template <bool FP8>
__device__ __forceinline__ float bound_value(const uint8_t *row, int d) {
    if constexpr (FP8) return e4m3x2_to_float2(row[d]).x;
    else return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[d]);
}

// The 8 bf16 or 16 E4M3 values of 16 bytes.
template <bool FP8>
__device__ __forceinline__ void unpack16(const uint4 &raw, float (&f)[FP8 ? 16 : 8]) {
    if constexpr (FP8) {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = e4m3x2_to_float2(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    } else {
        unpack_bf16x8(raw, f);
    }
}

// The pass reads 2 head_dim elements a page and multiplies each once: streaming them is its
// bound, so every SM holds 24 warps with up to 8 KB of bounds on their way each, and what comes
// before the stream is paid once: the (sequence, kv head, group of pages) steps form a line
// and every warp takes an equal run of it, with the next group's bounds sent for while one is
// multiplied and the page ids of the one after it.  29 us for 140 MB of bounds (8 sequences of
// 32k-131k tokens, 8 kv heads), 7 us of them the launch, the lengths and the last groups.  (A warp
// per 32 pages paid its two dependent reads and its query heads for every 16 KB: 37 us; bulk copies
// of single pages into shared memory were slower still, 47 us: 512 bytes are too little for one.)
// A page is UNITS units of 16 bytes (min row, then max row): 32 / UNITS pages a load, and the sums
// of a group's pages are reduced over the lanes at once by halving exchanges (9 shuffles for 8
// sums instead of 40).  Over 8-bit bounds the conversions are as long as the stream (20 us for 39 MB).
template <int HD, bool FP8>
struct ScoreCfg {
    static constexpr int PAGE = 2 * HD * (FP8 ? 1 : 2);
    static constexpr int UNITS = PAGE / 16;
    static constexpr int LANES = UNITS < 32 ? UNITS : 32;
    static constexpr int PARTS = UNITS / LANES;          // units a lane takes of a page
    static constexpr int PER = 32 / LANES;               // pages of a load
    static constexpr int LOADS = 8 / PARTS;              // page loads of a group: 4 KB
    static constexpr int GROUP = LOADS * PER;            // pages of a group
};

constexpr int kLeastGroup = 4;     // of any ScoreCfg
constexpr int kScoreThreads = 256;
constexpr size_t kScoreSmem = kScoreThreads * 2 * 8 * 16;   // two groups' bounds per warp
constexpr int kScoreSeqs = 512;    // sequences per launch (their prefix is in shared memory)

template <int HD, bool FP8>
__global__ void __launch_bounds__(kScoreThreads, 3) score_kernel(const __grid_constant__ SelectParams p) {
    using C = ScoreCfg<HD, FP8>;
    static_assert(C::GROUP >= kLeastGroup && C::GROUP <= 32, "group");
    constexpr int UNITS = C::UNITS, LANES = C::LANES, PARTS = C::PARTS, PER = C::PER, LOADS = C::LOADS;
    constexpr int E = FP8 ? 16 : 8;               // elements of a unit
    extern __shared__ __align__(16) uint32_t dyn[];
    __shared__ int64_t pref[kScoreSeqs + 1];      // groups before sequence b
    __shared__ int pages[kScoreSeqs];
    __shared__ int64_t even;                      // groups of a warp's run
    __shared__ int more;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int b = threadIdx.x; b < p.num_seqs; b += kScoreThreads) {
        const int np = (select_len(p, b, false) + kBlockSize - 1) / kBlockSize;
        pages[b] = np;
        pref[b + 1] = np > p.max_pages ? static_cast<int64_t>((np + C::GROUP - 1) / C::GROUP) * p.nkv : 0;
    }
    if (threadIdx.x == 0) pref[0] = 0;
    __syncthreads();
    if (warp == 0) {
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
        if (lane == 0) {
            const int n_warps = static_cast<int>(gridDim.x) * (kScoreThreads / 32);
            even = carry / n_warps;
            more = static_cast<int>(carry - even * n_warps);
        }
    }
    __syncthreads();
    // neighbouring runs go to different SMs; the first `more` runs are one group longer
    const int me = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    int64_t u = even * me + min(me, more);
    const int64_t end = u + even + (me < more ? 1 : 0);
    if (u >= end) return;
    int b = 0;
    for (int hi = p.num_seqs; hi - b > 1;) {      // the largest b with pref[b] <= u
        const int mid = (b + hi) >> 1;
        if (pref[mid] <= u) b = mid; else hi = mid;
    }
    auto groups_of = [&](int b) { return (pages[b] + C::GROUP - 1) / C::GROUP; };
    const int64_t in = u - pref[b];               // below nkv groups
    int kh = in <= INT32_MAX ? static_cast<int>(in) / groups_of(b) : static_cast<int>(in / groups_of(b));
    int grp = static_cast<int>(in - static_cast<int64_t>(kh) * groups_of(b));
    const int unit = lane % LANES, sub = lane / LANES;
    const int g = p.nq / p.nkv;
    auto page_id = [&](int b, int grp) -> int {
        const int i = grp * C::GROUP + lane;
        return lane < C::GROUP && i < pages[b] ? p.block_tables[static_cast<int64_t>(b) * p.max_blocks + i] : 0;
    };
    auto advance = [&](int &b, int &kh, int &grp) {
        if (++grp < groups_of(b)) return;
        grp = 0;
        if (++kh < p.nkv) return;
        kh = 0;
        do ++b; while (b + 1 < p.num_seqs && pref[b + 1] == pref[b]);
    };
    // Sends a group's bounds to this lane's places of a stage; the pages with ids out of range.
    uint4 *ring = reinterpret_cast<uint4 *>(dyn) + warp * (2 * 8 * 32) + lane;
    auto send = [&](int stage, int b, int kh, int grp, int id) -> unsigned {
        const bool known = id >= 0 && id < p.num_blocks;
        if (!known) atomicOr(p.status, kStatusBounds);
        // lane i knows where page i's bounds are, in units of 16 bytes (the host sees to it that 32
        // bits hold them).  Pages that are not ranked (the first ones, the newest, those past the end)
        // take the group's first ranked one's: their own may hold anything, and S is not to know.
        const int from = max(p.sink - grp * C::GROUP, 0), past = pages[b] - p.recent - grp * C::GROUP;
        const int whose = lane >= from && lane < past ? lane : from;
        const uint32_t place = (static_cast<uint32_t>(__shfl_sync(kAll, known ? id : 0, whose < C::GROUP ? whose : 0)) * p.nkv + kh) * UNITS;
        const uint4 *src = reinterpret_cast<const uint4 *>(p.bounds) + unit;
#pragma unroll
        for (int k = 0; k < LOADS; ++k) {
            const uint32_t at = __shfl_sync(kAll, place, k * PER + sub);
#pragma unroll
            for (int v = 0; v < PARTS; ++v)
                cp_async_16(ring + (stage * 8 + k * PARTS + v) * 32, src + (at + v * LANES));
        }
        return __ballot_sync(kAll, !known);
    };
    int stage = 0;
    unsigned unknown = send(0, b, kh, grp, page_id(b, grp));
    cp_async_commit();
    int b1 = b, kh1 = kh, grp1 = grp;             // the next group, and its ids
    advance(b1, kh1, grp1);
    int id1 = u + 1 < end ? page_id(b1, grp1) : 0;
    float w[PARTS][E];   // this lane's weights: N for the units of the min row (a page's first half), else P
    for (bool fresh = true; u < end; ++u) {
        unsigned unknown1 = 0;
        int b2 = b1, kh2 = kh1, grp2 = grp1, id2 = 0;
        if (u + 1 < end) {
            unknown1 = send(stage ^ 1, b1, kh1, grp1, id1);
            advance(b2, kh2, grp2);
            if (u + 2 < end) id2 = page_id(b2, grp2);
        }
        cp_async_commit();
        const int first = grp * C::GROUP, n = min(C::GROUP, pages[b] - first);
        const int64_t row = static_cast<int64_t>(b) * p.nkv + kh;
        if (fresh) {
#pragma unroll
            for (int v = 0; v < PARTS; ++v) {
                const int at = v * LANES + unit;
                const bool low = at < UNITS / 2;
                const __nv_bfloat16 *q = p.q + (static_cast<int64_t>(b) * p.nq + kh * g) * HD +
                                         (low ? at : at - UNITS / 2) * E;
#pragma unroll
                for (int e = 0; e < E; ++e) w[v][e] = 0.f;
#pragma unroll 4
                for (int h = 0; h < g; ++h) {
#pragma unroll
                    for (int e0 = 0; e0 < E; e0 += 8) {
                        // max(q, 0), or max(-q, 0) for N; a NaN stays one
                        uint4 raw8 = *reinterpret_cast<const uint4 *>(q + static_cast<int64_t>(h) * HD + e0);
                        const uint32_t turn = low ? 0x80008000u : 0u;
                        raw8.x = max2<false>(raw8.x ^ turn, 0u), raw8.y = max2<false>(raw8.y ^ turn, 0u);
                        raw8.z = max2<false>(raw8.z ^ turn, 0u), raw8.w = max2<false>(raw8.w ^ turn, 0u);
                        float f[8];
                        unpack_bf16x8(raw8, f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[v][e0 + e] += f[e];
                    }
                }
                if (low)
#pragma unroll
                    for (int e = 0; e < E; ++e) w[v][e] = -w[v][e];
            }
        }
        cp_async_wait<1>();     // this group's bounds are here; a lane reads what it sent for
        const uint4 *raw = ring + stage * 8 * 32;
        float x[LOADS];         // the pages' sums
        float far[PARTS][E];    // the largest magnitudes of the group's elements
        bool odd = false;
#pragma unroll
        for (int k = 0; k < LOADS; k += 2) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int v = 0; v < PARTS; ++v) {
                float f[2][E];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    unpack16<FP8>(raw[((k + u) * PARTS + v) * 32], f[u]);
                    float2 c[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};   // chains of E / 4 products
#pragma unroll
                    for (int e = 0; e < E; e += 2)
                        c[e / 2 & 1] = __ffma2_rn(make_float2(w[v][e], w[v][e + 1]), make_float2(f[u][e], f[u][e + 1]),
                                                  c[e / 2 & 1]);
                    const float2 c2 = __fadd2_rn(c[0], c[1]);
                    s[u] += c2.x + c2.y;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) far[v][e] = most_of(k ? far[v][e] : 0.f, f[0][e], f[1][e]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                x[k + u] = s[u];
                odd |= s[u] != s[u];
            }
        }
        if (odd) {   // a zero weight met an infinity, or a sum is a NaN: the exact rule
#pragma unroll 1
            for (int k = 0; k < LOADS; ++k) {
                float y = 0.f;
#pragma unroll
                for (int v = 0; v < PARTS; ++v) {
                    float f[E];
                    unpack16<FP8>(raw[(k * PARTS + v) * 32], f);
#pragma unroll
                    for (int e = 0; e < E; ++e) y += weighed(w[v][e], f[e]);
                }
#pragma unroll
                for (int j = 0; j < LOADS; ++j) x[j] = j == k ? y : x[j];
            }
        }
        float most = 0.f;   // S of a page with the group's largest magnitudes
#pragma unroll
        for (int v = 0; v < PARTS; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e) most += weighed(fabsf(w[v][e]), far[v][e]);
        __syncwarp();
        int which = 0;   // the sum this lane ends up with
        int m = LANES / 2;
#pragma unroll
        for (int half = LOADS / 2; half >= 1; half >>= 1, m >>= 1) {
            const bool up = lane & m;
            which += up ? half : 0;
#pragma unroll
            for (int i = 0; i < LOADS / 2; ++i)
                if (i < half) {
                    const float give = up ? x[i] : x[i + half];
                    x[i] = (up ? x[i + half] : x[i]) + __shfl_xor_sync(kAll, give, m);
                }
        }
#pragma unroll
        for (int o = LANES / (2 * LOADS); o >= 1; o >>= 1) x[0] += __shfl_xor_sync(kAll, x[0], o);
        const int i = which * PER + sub;
        if (unit % (LANES / LOADS) == 0 && i < n)
            p.score[row * p.max_blocks + first + i] = unknown >> i & 1 ? -INFINITY : x[0];
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float y = __shfl_xor_sync(kAll, most, o);
            most = o < LANES ? most + y : max_nan(most, y);
        }
        const bool ranked = max(p.sink, first) < min(pages[b] - p.recent, first + C::GROUP);
        if (lane == 0) p.span[row * p.groups + grp] = ranked ? most : 0.f;
        fresh = kh1 != kh || b1 != b;
        b = b1, kh = kh1, grp = grp1;
        b1 = b2, kh1 = kh2, grp1 = grp2;
        unknown = unknown1;
        id1 = id2;
        stage ^= 1;
    }
}

// ---- selection ------------------------------------------------------------------------------

// Order-preserving whole numbers of floating scores; a NaN is the largest.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (isnan(x)) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float score_of(uint32_t k) {
    return k == 0xffffffffu ? NAN : __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ uint64_t key_of(double x) {
    if (isnan(x)) return ~0ull;
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x == 0.0 ? 0.0 : x));
    return u >> 63 ? ~u : u | 1ull << 63;
}

// Sums of three counts over the CTA's NT threads; sh holds two halves, used in turn.
template <int NT>
struct BlockSums {
    static constexpr int W = NT / 32;
    int *sh;   // [2][3][32]
    int turn;
    __device__ __forceinline__ void operator()(int (&x)[3]) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int *at = sh + turn * 96;
        turn ^= 1;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int v = __reduce_add_sync(kAll, x[i]);
            if (lane == 0) at[i * 32 + warp] = v;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 3; ++i) x[i] = __reduce_add_sync(kAll, lane < W ? at[i * 32 + lane] : 0);
    }
};

// The f-th largest (f >= 1) of the keys that count(t, c) counts (c += this thread's keys that
// are >= t): the largest t with at least f keys >= t, found two bits at a time below `shift`;
// `t` holds the bits from `shift` on, which the f-th largest is known to have.
template <typename Key, typename Sums, typename Count>
__device__ __forceinline__ Key nth_largest(Key t, int shift, int f, Sums &sums, Count count) {
    for (shift -= 2; shift >= 0; shift -= 2) {
        int c[3] = {0, 0, 0};
#pragma unroll
        for (int i = 0; i < 3; ++i) count(static_cast<Key>(t | static_cast<Key>(i + 1) << shift), c[i]);
        sums(c);
        const int digit = c[2] >= f ? 3 : (c[1] >= f ? 2 : (c[0] >= f ? 1 : 0));
        t |= static_cast<Key>(digit) << shift;
    }
    return t;
}

// Exclusive prefix of x over the CTA's NT threads, and the total.
template <int NT>
__device__ __forceinline__ int block_scan(int x, int *warps, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = v;
    __syncthreads();
    const int w = lane < NT / 32 ? warps[lane] : 0;
    total = __reduce_add_sync(kAll, w);
    return __reduce_add_sync(kAll, lane < warp ? w : 0) + v - x;
}

constexpr int kBins = 2048;
constexpr int kFew = 32;                       // pages at the border that one warp puts in order
constexpr int kShortPages = 1024;              // tables for fewer threads
constexpr int kHeldPages = 40960;              // pages whose scores fit shared memory
constexpr int kMostPages = 1 << 19;            // pages whose outcome bits do
constexpr int kBatch = 8;                      // pages a thread takes at once

// Scores held for n pages: whole batches of the CTA's threads, so that no pass checks its ends.
__host__ __device__ inline int select_held(int n, int threads) {
    return (n + threads * kBatch - 1) / (threads * kBatch) * (threads * kBatch);
}

// Bytes of dynamic shared memory: scores (HELD), then three words per 32 pages.
size_t select_smem(int max_blocks, int threads, bool held) {
    return (held ? static_cast<size_t>(select_held(max_blocks, threads)) * 4 : 0) +
           static_cast<size_t>((max_blocks + 31) / 32) * 12;
}

// One CTA per (kv head, sequence); all passes go over the pages in the same order, thread t
// taking pages t, t + NT, ...  The border score's bin comes from a histogram of even bins over the
// scores' range (scores crowd in few binades, so bins of their bits would not part them).  One more
// pass then settles every page whose score is 2E away from that bin; the few others are put in
// order, by exact scores where 2E does not part them, and join.  Where more than 32 pages are that
// close to the border, or scores are not finite, the border is found by counting instead, two bits
// a step below the bits that all candidates share.  A page's outcome is a bit of its warp's word;
// one scan over the words' counts gives every chosen page its place, in page order.  A row is one
// chain of dependent steps, bound by their latency and by what its SM can issue, not by its 32 KB of
// scores: passes take eight scores a thread at once, all read before any is used (one after another
// they cost 11800 of a row's 31600 cycles in the first pass alone).  A row of 131072 tokens takes
// 14000 cycles, 64 rows 15 us; with passes of their own for the border's pages, the band around it
// and every page's outcome they took 27500 and 21.
template <int HD, bool FP8, int NT, bool HELD>
__global__ void __launch_bounds__(NT) select_kernel(const __grid_constant__ SelectParams p) {
    constexpr int ROW = HD * (FP8 ? 1 : 2);
    constexpr int W = NT / 32;
    extern __shared__ uint32_t dyn[];
    __shared__ int sums_sh[2 * 3 * 32];
    __shared__ int warps[32];
    __shared__ uint32_t ends[3][32];
    __shared__ double P[HD], N[HD];
    __shared__ int hist[kBins];
    __shared__ float few_x[kFew];
    __shared__ uint64_t few_key[kFew];
    __shared__ int few_page[kFew];
    __shared__ int bin_at, bin_above, near_n, few_n;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int kh = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = select_len(p, b, kh == 0 && tid == 0);
    const int np = (L + kBlockSize - 1) / kBlockSize;
    const int kept = min(np, p.max_pages);
    const int64_t row = static_cast<int64_t>(b) * p.nkv + kh;
    const int32_t *bt = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
    int32_t *out = p.page_tables + row * p.max_pages;
    if (kh == 0 && tid == 0) p.page_lens[b] = kept * kBlockSize - (np * kBlockSize - L);
    for (int i = kept + tid; i < p.max_pages; i += NT) out[i] = -1;
    if (np <= p.max_pages) {   // no score pass has seen these pages' ids
        for (int i = tid; i < np; i += NT) {
            const int id = bt[i];
            out[i] = id;
            if (id < 0 || id >= p.num_blocks) atomicOr(p.status, kStatusBounds);
        }
        return;
    }
    // f of the candidates [lo, hi) join the sinks and the newest pages
    const int lo = p.sink, hi = np - p.recent, f = p.max_pages - p.sink - p.recent;
    const float *score = p.score + row * p.max_blocks;
    float *held_x = reinterpret_cast<float *>(dyn);
    const int held = select_held(np, NT);
    uint32_t *words = dyn + (HELD ? select_held(p.max_blocks, NT) : 0); // outcome bits of 32 pages
    const int n_words = (np + 31) / 32;
    uint32_t *tie_words = words + (p.max_blocks + 31) / 32;
    auto candidate = [&](int i) { return static_cast<unsigned>(i - lo) < static_cast<unsigned>(hi - lo); };
    // a candidate's score, infinity for pages that are chosen anyway, and -infinity past the pages
    auto read_x = [&](int i) { return candidate(i) ? score[i] : (i < np ? INFINITY : -INFINITY); };
    // calls f(page, score) for this thread's pages, a batch of scores read before any call
    auto each_x = [&](auto f) {
        for (int i0 = tid; i0 < held; i0 += NT * kBatch) {
            float x[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) x[u] = HELD ? held_x[i0 + u * NT] : read_x(i0 + u * NT);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) f(i0 + u * NT, x[u]);
        }
    };
    // page i's score in fp64, by one warp, from P and N
    auto exact_weights = [&]() {
        const int g = p.nq / p.nkv;
        for (int d = tid; d < HD; d += NT) {
            const __nv_bfloat16 *q = p.q + (static_cast<int64_t>(b) * p.nq + kh * g) * HD + d;
            double x = 0.0, y = 0.0;
#pragma unroll 8
            for (int h = 0; h < g; ++h) {
                const float v = __bfloat162float(q[h * HD]);
                if (v < 0.f) y += v;
                else x += v;
            }
            P[d] = x;
            N[d] = y;
        }
        __syncthreads();
    };
    auto exact_score = [&](int i) -> double {
        const int id = bt[i];
        if (id < 0 || id >= p.num_blocks) return -INFINITY;
        const uint8_t *r = p.bounds + (static_cast<int64_t>(id) * p.nkv + kh) * 2 * ROW;
        double e = 0.0;
#pragma unroll
        for (int d = 0; d < HD; d += 32)
            e += weighed<double>(P[d + lane], bound_value<FP8>(r + ROW, d + lane)) +
                 weighed<double>(N[d + lane], bound_value<FP8>(r, d + lane));
#pragma unroll
        for (int o = 16; o; o >>= 1) e += __shfl_xor_sync(kAll, e, o);
        return e;
    };
    BlockSums<NT> sums{sums_sh, 0};
    float least = INFINITY, top = -INFINITY, span = 0.f;   // ends of the scores; S of the bound E
    bool odd = f == 0;                                     // a score is not finite, or none is asked for
    if (f > 0) {
        for (int i0 = tid; i0 < held; i0 += NT * kBatch) {
            float x[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) x[u] = read_x(i0 + u * NT);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u * NT;
                if constexpr (HELD) held_x[i] = x[u];
                least = fminf(least, candidate(i) ? x[u] : INFINITY);
                top = fmaxf(top, candidate(i) ? x[u] : -INFINITY);
                odd |= candidate(i) && !(fabsf(x[u]) < INFINITY);
            }
        }
        const float *spans = p.span + row * p.groups;
        const int n_spans = (np + p.group - 1) / p.group;
        for (int i0 = tid; i0 < n_spans; i0 += NT * 4) {
            float x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = i0 + u * NT < n_spans ? spans[i0 + u * NT] : 0.f;
            span = max_nan(span, max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])));
        }
    }
    for (int i = tid; i < kBins; i += NT) hist[i] = 0;
    if (tid == 0) near_n = few_n = 0;
    const uint32_t k_least = __reduce_min_sync(kAll, key_of(least)), k_top = __reduce_max_sync(kAll, key_of(top));
    const uint32_t k_span = __reduce_max_sync(kAll, key_of(span));   // a NaN is the largest
    if (lane == 0) ends[0][warp] = k_least, ends[1][warp] = k_top, ends[2][warp] = k_span;
    odd = __syncthreads_or(odd);
    least = score_of(__reduce_min_sync(kAll, lane < W ? ends[0][lane] : 0xffffffffu));
    top = score_of(__reduce_max_sync(kAll, lane < W ? ends[1][lane] : 0u));
    span = score_of(__reduce_max_sync(kAll, lane < W ? ends[2][lane] : 0u));
    const float E2 = 2.f * static_cast<float>(p.nq / p.nkv + 24) * 0x1p-24f * span + 0x1p-138f;
    const float scale = (kBins - 1) / (top - least);
    // a score's place among the bins, rounded by less than 2^-12; 2E there, with both roundings
    auto place_of = [&](float x) { return (x - least) * scale; };
    const float margin = E2 * scale + 0x1p-10f;
    bool settled = !odd && scale > 0.f && margin < 8.f;   // not for an infinite or NaN scale either
    if (settled) {
        each_x([&](int, float x) {
            if (fabsf(x) < INFINITY) atomicAdd(&hist[static_cast<int>(place_of(x))], 1);
        });
        __syncthreads();
        constexpr int EACH = kBins / NT;
        const int first_bin = kBins - 1 - tid * EACH;   // from the top, EACH bins a thread
        int c = 0, total;
#pragma unroll
        for (int i = 0; i < EACH; ++i) c += hist[first_bin - i];
        int before = block_scan<NT>(c, warps, total);
        if (before < f && f <= before + c) {
            int at = first_bin;
            while (before + hist[at] < f) before += hist[at--];
            bin_at = at;
            bin_above = before;
        }
        __syncthreads();
        const int bin = bin_at;
        const float from = bin - margin, past = bin + 1 + margin;
        each_x([&](int i, float x) {
            const float y = place_of(x);
            const unsigned w = __ballot_sync(kAll, y >= past);
            if (lane == 0 && i < np) words[i / 32] = w;
            if (y >= from && y < past) {
                const int at = atomicAdd(&near_n, 1);
                if (at < kFew) few_x[at] = x, few_page[at] = i;
            }
        });
        __syncthreads();
        const int m = near_n;
        settled = m <= kFew;
        if (settled) {   // every warp puts the m pages at the border in order
            const bool here = lane < m;
            const float x = here ? few_x[lane] : 0.f;
            const int page = here ? few_page[lane] : 0;
            // winners among them: pages of higher bins are counted in bin_above
            const int need = f - bin_above + __popc(__ballot_sync(kAll, here && static_cast<int>(place_of(x)) > bin));
            int rank = 0;
            for (int i = 0; i < m; ++i) {
                const float o = __shfl_sync(kAll, x, i);
                rank += o > x || (o == x && i < lane);
            }
            const float T = __shfl_sync(kAll, x, __ffs(__ballot_sync(kAll, here && rank == need - 1)) - 1);
            bool win = here && x > T + E2;
            const bool band = here && !win && x >= T - E2;
            const unsigned in_band = __ballot_sync(kAll, band);
            const int take = need - __popc(__ballot_sync(kAll, win));
            if (take == __popc(in_band)) {
                win |= band;
            } else {
                exact_weights();
                for (int i = warp; i < m; i += W)
                    if (in_band >> i & 1) {
                        const double e = exact_score(few_page[i]);
                        if (lane == 0) few_key[i] = key_of(e);
                    }
                __syncthreads();
                const uint64_t k = band ? few_key[lane] : 0ull;
                int place = 0;   // of the band's pages, by (score, page)
                for (unsigned r = in_band; r; r &= r - 1) {
                    const int i = __ffs(r) - 1;
                    const uint64_t o = few_key[i];
                    place += o > k || (o == k && few_page[i] < page);
                }
                win |= band && place < take;
            }
            if (warp == 0 && win) atomicOr(&words[page / 32], 1u << (page & 31));
            __syncthreads();
        }
    }
    if (!settled) {
        auto key_at = [&](int i, float x) -> uint32_t { return f > 0 && candidate(i) ? key_of(x) : 0u; };
        // calls f(page, key) for this thread's pages; 0 for pages that are not candidates
        auto each_key = [&](auto f) { each_x([&](int i, float x) { f(i, key_at(i, x)); }); };
        // Keys of the sure winners (> above) and of the sure losers (< below); the band between.
        uint32_t above = 0xffffffffu, below = 0xffffffffu;
        bool all = true;                            // the whole band wins
        uint64_t edge = 0;                          // else the weakest exact score that wins ...
        int ties = 0;                               // ... and how many equal to it do
        double *exact = p.exact + row * p.max_blocks;
        if (f > 0) {
            const uint32_t best = key_of(top);
            const int bits = odd ? 32 : (32 - __clz(key_of(least) ^ best) + 1) & ~1;   // below the shared ones, even
            const uint32_t t = nth_largest<uint32_t>(bits == 32 ? 0u : best >> bits << bits, bits, f, sums, [&](uint32_t x, int &c) {
                each_key([&](int, uint32_t k) { c += k >= x; });
            });
            const float T = score_of(t);
            if (isfinite(E2) && !isnan(T)) {   // else nothing is sure and all are in the band
                above = key_of(T + E2);
                below = key_of(T - E2);
            } else {
                below = 1u;
            }
            int c[3] = {0, 0, 0};
            each_key([&](int, uint32_t k) {
                c[0] += k > above;
                c[1] += k >= below && k <= above;
            });
            sums(c);
            const int take = f - c[0];   // winners that come from the band
            all = take == c[1];
            if (!all) {
                exact_weights();
                for (int base = warp * 32; base < np; base += NT) {
                    const int mine = base + lane;
                    const uint32_t k = mine < np ? key_at(mine, HELD ? held_x[mine] : read_x(mine)) : 0u;
                    for (unsigned m = __ballot_sync(kAll, k >= below && k <= above); m; m &= m - 1) {
                        const int i = base + __ffs(m) - 1;
                        const double e = exact_score(i);
                        if (lane == 0) exact[i] = e;
                    }
                }
                __syncthreads();
                auto count = [&](uint64_t x, int &n, bool strict) {
                    each_key([&](int i, uint32_t k) {
                        if (k < below || k > above) return;
                        const uint64_t e = key_of(exact[i]);
                        n += strict ? e > x : e >= x;
                    });
                };
                edge = nth_largest<uint64_t>(0ull, 64, take, sums, [&](uint64_t x, int &n) { count(x, n, false); });
                int n[3] = {0, 0, 0};
                count(edge, n[0], true);
                sums(n);
                ties = take - n[0];
            }
        }
        each_key([&](int i, uint32_t k) {
            bool win = (i < np && !candidate(i)) || k > above, tie = false;
            if (!win && k && k >= below) {   // in the band
                const uint64_t e = all ? 1ull : key_of(exact[i]);
                win = all || e > edge;
                tie = !all && e == edge;
            }
            const unsigned w = __ballot_sync(kAll, win), t = __ballot_sync(kAll, tie);
            if (lane == 0 && i < np) {
                words[i / 32] = w;
                tie_words[i / 32] = t;
            }
        });
        __syncthreads();
        if (!all) {   // of the pages that tie at the edge, the lowest `ties` win
            const int each = (n_words + NT - 1) / NT, w0 = min(tid * each, n_words), w1 = min(w0 + each, n_words);
            int n = 0, total;
            for (int i = w0; i < w1; ++i) n += __popc(tie_words[i]);
            int left = ties - block_scan<NT>(n, warps, total);
            for (int i = w0; i < w1 && left > 0; ++i)
                for (uint32_t t = tie_words[i]; t && left > 0; t &= t - 1, --left) words[i] |= t & -t;
        }
    }
    // every thread takes `each` consecutive words
    const int each = (n_words + NT - 1) / NT, w0 = min(tid * each, n_words), w1 = min(w0 + each, n_words);
    int n = 0, total;
    for (int i = w0; i < w1; ++i) n += __popc(words[i]);
    int at = block_scan<NT>(n, warps, total);
    if constexpr (HELD) {
        // The winners' numbers first (over the scores, which have done their work), so that each
        // thread then waits for one block-table read and not for one per winner of its words.
        int *won = reinterpret_cast<int *>(held_x);
        for (int i = w0; i < w1; ++i)
            for (uint32_t w = words[i]; w; w &= w - 1) won[at++] = i * 32 + __ffs(w) - 1;
        __syncthreads();
#pragma unroll 4
        for (int i = tid; i < kept; i += NT) out[i] = bt[won[i]];
    } else {
        int *places = reinterpret_cast<int *>(tie_words + (p.max_blocks + 31) / 32);
        for (int i = w0; i < w1; ++i) {
            places[i] = at;
            at += __popc(words[i]);
        }
        __syncthreads();
        for (int base = warp * 32; base < np; base += NT) {
            const uint32_t w = words[base / 32];
            if (w >> lane & 1) out[places[base / 32] + __popc(w & ((1u << lane) - 1))] = bt[base + lane];
        }
    }
}

template <int HD, bool FP8>
cudaError_t launch_select(SelectParams &p, cudaStream_t stream) {
    using C = ScoreCfg<HD, FP8>;
    p.group = C::GROUP;
    p.groups = (p.max_blocks + C::GROUP - 1) / C::GROUP;
    static std::atomic<int> configured{-1};   // last device whose attributes are set
    static std::atomic<int> sm_count{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    auto allow = [&](auto kern, int pages, int threads, bool held) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(select_smem(pages, threads, held)));
    };
    if (configured.load() != dev) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(score_kernel<HD, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreSmem);
        allow(select_kernel<HD, FP8, 256, true>, kShortPages, 256, true);
        allow(select_kernel<HD, FP8, 512, true>, kHeldPages, 512, true);
        allow(select_kernel<HD, FP8, 512, false>, kMostPages, 512, false);
        if (e != cudaSuccess) return e;
        sm_count = n;
        configured = dev;
    }
    if (p.max_blocks > p.max_pages) {
        // three CTAs an SM, or a warp for every group there can be
        const int64_t most = (static_cast<int64_t>(p.num_seqs) * p.nkv * p.groups + 7) / 8;
        const int64_t room = 3 * sm_count.load();
        const unsigned grid = static_cast<unsigned>(most < room ? most : room);
        e = launch_after(score_kernel<HD, FP8>, dim3(grid), kScoreThreads, p, stream, kScoreSmem);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid(p.nkv, p.num_seqs);
    auto select = [&](auto kern, int threads, bool held) {
        return launch_after(kern, grid, threads, p, stream, select_smem(p.max_blocks, threads, held));
    };
    // short tables: fewer warps to wait for at each barrier
    if (p.max_blocks <= kShortPages) return select(select_kernel<HD, FP8, 256, true>, 256, true);
    if (p.max_blocks <= kHeldPages) return select(select_kernel<HD, FP8, 512, true>, 512, true);
    return select(select_kernel<HD, FP8, 512, false>, 512, false);
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Offsets of the workspace's parts (scores, spans, exact scores) and its size.
size_t select_layout(int num_seqs, int nkv, int max_blocks, size_t off[3]) {
    const size_t rows = static_cast<size_t>(num_seqs > 0 ? num_seqs : 0) * (nkv > 0 ? nkv : 0);
    const size_t n = rows * (max_blocks > 0 ? max_blocks : 0);
    const size_t groups = (static_cast<size_t>(max_blocks > 0 ? max_blocks : 0) + kLeastGroup - 1) / kLeastGroup;
    off[0] = 0;
    off[1] = off[0] + round256(n * 4);
    off[2] = off[1] + round256(rows * groups * 4);
    return off[2] + round256(n * 8);
}

}  // namespace
}  // namespace pa

extern "C" int pa_page_bounds(void *bounds, const void *k_cache, const int32_t *block_tables,
                              const int32_t *seq_lens, const int32_t *first_tokens,
                              int max_new_tokens, int num_seqs, int num_kv_heads, int head_dim,
                              int block_size, int max_blocks_per_seq, int64_t num_blocks,
                              int64_t stride_block, int64_t stride_head, int64_t stride_token,
                              int kv_dtype, void *stream) {
    using namespace pa;
    if (num_seqs < 0 || max_new_tokens < 0)
        return api_fail(PA_ERR_INVALID, "num_seqs %d, max_new_tokens %d", num_seqs, max_new_tokens);
    int rc = api_check_heads(head_dim, num_kv_heads, num_kv_heads);
    if (rc) return rc;
    rc = api_check_kv_dtype(kv_dtype, 1.f, 1.f);
    if (rc) return rc;
    rc = api_check_pool(head_dim, block_size, num_blocks, num_kv_heads, stride_block, stride_head,
                        stride_token, kv_dtype);
    if (rc) return rc;
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > INT32_MAX / kBlockSize)
        return api_fail(PA_ERR_INVALID, "max_blocks_per_seq %d", max_blocks_per_seq);
    if (num_seqs == 0 || max_new_tokens == 0) return PA_OK;
    if (!bounds || !k_cache || !block_tables || !seq_lens)
        return api_fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned(bounds, 16) || !aligned(k_cache, 16))
        return api_fail(PA_ERR_INVALID, "bounds and the key pool must be 16-byte aligned");
    // pages that max_new_tokens tokens can touch: one more when they start inside a page
    const int64_t touched = (static_cast<int64_t>(max_new_tokens) + (first_tokens ? 2 : 1) * (kBlockSize - 1)) / kBlockSize;
    const int pages = static_cast<int>(touched < max_blocks_per_seq ? touched : max_blocks_per_seq);
    if (static_cast<int64_t>(num_seqs) * pages * num_kv_heads / 8 >= INT32_MAX ||
        static_cast<int64_t>(pages) * num_kv_heads > INT32_MAX)   // the kernel counts a sequence's in 32 bits
        return api_fail(PA_ERR_UNSUPPORTED, "too many pages for one launch");
    const int elem = kv_dtype == PA_KV_FP8_E4M3 ? 1 : 2;
    BoundsParams p = {};
    p.bounds = static_cast<uint8_t *>(bounds);
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.first_tokens = first_tokens;
    p.num_blocks = num_blocks;
    p.b_block = stride_block * elem;
    p.b_head = stride_head * elem;
    p.b_token = stride_token * elem;
    p.num_seqs = num_seqs;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.pages = pages;
    rc = api_status_ptr(&p.status);
    if (rc) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fp8 = elem == 1;
    const cudaError_t e = head_dim == 64    ? launch_bounds<64>(p, fp8, s)
                          : head_dim == 128 ? launch_bounds<128>(p, fp8, s)
                                            : launch_bounds<256>(p, fp8, s);
    if (e != cudaSuccess) return api_cuda_fail(e, "page bounds launch");
    return PA_OK;
}

extern "C" size_t pa_select_pages_workspace_size(int num_seqs, int num_kv_heads,
                                                 int max_blocks_per_seq) {
    size_t off[3];
    return pa::select_layout(num_seqs, num_kv_heads, max_blocks_per_seq, off);
}

extern "C" int pa_select_pages(int32_t *page_tables, int32_t *page_lens, const void *q,
                               const void *bounds, const int32_t *block_tables,
                               const int32_t *seq_lens, int num_seqs, int num_q_heads,
                               int num_kv_heads, int head_dim, int block_size,
                               int max_blocks_per_seq, int64_t num_blocks, int max_pages,
                               int sink_pages, int recent_pages, int kv_dtype, void *workspace,
                               size_t workspace_bytes, void *stream) {
    using namespace pa;
    if (num_seqs < 0) return api_fail(PA_ERR_INVALID, "num_seqs %d", num_seqs);
    int rc = api_check_heads(head_dim, num_q_heads, num_kv_heads);
    if (rc) return rc;
    rc = api_check_kv_dtype(kv_dtype, 1.f, 1.f);
    if (rc) return rc;
    if (block_size != kBlockSize)
        return api_fail(PA_ERR_UNSUPPORTED, "block_size %d: only 16-token blocks", block_size);
    if (num_blocks <= 0) return api_fail(PA_ERR_INVALID, "num_blocks %lld", (long long)num_blocks);
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > INT32_MAX / kBlockSize)
        return api_fail(PA_ERR_INVALID, "max_blocks_per_seq %d", max_blocks_per_seq);
    if (max_blocks_per_seq > kMostPages)
        return api_fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq %d > %d", max_blocks_per_seq, kMostPages);
    if (max_pages <= 0 || max_pages > INT32_MAX / kBlockSize)
        return api_fail(PA_ERR_INVALID, "max_pages %d", max_pages);
    if (sink_pages < 0 || recent_pages < 1 || sink_pages > max_pages ||
        recent_pages > max_pages - sink_pages)
        return api_fail(PA_ERR_INVALID, "sink_pages %d and recent_pages %d (at least 1) in %d pages",
                        sink_pages, recent_pages, max_pages);
    if (num_seqs > 65535 || num_kv_heads > 65535)
        return api_fail(PA_ERR_UNSUPPORTED, "num_seqs %d, num_kv_heads %d: at most 65535", num_seqs,
                        num_kv_heads);
    if (num_blocks > (int64_t(1) << 32) / num_kv_heads / head_dim * (kv_dtype == PA_KV_FP8_E4M3 ? 8 : 4))
        return api_fail(PA_ERR_UNSUPPORTED, "num_blocks %lld: bounds of 2^32 16-byte units at most", (long long)num_blocks);
    if (num_seqs == 0) return PA_OK;
    if (!page_tables || !page_lens || !q || !bounds || !block_tables || !seq_lens)
        return api_fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned(q, 16) || !aligned(bounds, 16))
        return api_fail(PA_ERR_INVALID, "q and bounds must be 16-byte aligned");
    size_t off[3];
    const size_t need = select_layout(num_seqs, num_kv_heads, max_blocks_per_seq, off);
    if (workspace_bytes < need)
        return api_fail(PA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (!workspace || !aligned(workspace, 256))
        return api_fail(PA_ERR_WORKSPACE, "workspace must be non-null and 256-byte aligned");
    const int64_t listed = static_cast<int64_t>(num_seqs) * num_kv_heads * max_pages;
    const int64_t tables = static_cast<int64_t>(num_seqs) * max_blocks_per_seq;
    if (api_overlap(page_lens, num_seqs, seq_lens, num_seqs) || api_overlap(page_lens, num_seqs, block_tables, tables) ||
        api_overlap(page_tables, listed, seq_lens, num_seqs) || api_overlap(page_tables, listed, block_tables, tables) ||
        api_overlap(page_tables, listed, page_lens, num_seqs))
        return api_fail(PA_ERR_INVALID, "page_lens and page_tables must not overlap seq_lens, block_tables or one another");
    char *ws = static_cast<char *>(workspace);
    SelectParams p = {};
    p.page_tables = page_tables;
    p.page_lens = page_lens;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.bounds = static_cast<const uint8_t *>(bounds);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.score = reinterpret_cast<float *>(ws + off[0]);
    p.span = reinterpret_cast<float *>(ws + off[1]);
    p.exact = reinterpret_cast<double *>(ws + off[2]);
    p.num_blocks = num_blocks;
    p.num_seqs = num_seqs;
    p.nq = num_q_heads;
    p.nkv = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.max_pages = max_pages;
    p.sink = sink_pages;
    p.recent = recent_pages;
    rc = api_status_ptr(&p.status);
    if (rc) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
    // the score pass holds kScoreSeqs sequences' lengths: more go in several launches
    for (int at = 0; at < num_seqs; at += kScoreSeqs) {
        SelectParams a = p;
        a.num_seqs = num_seqs - at < kScoreSeqs ? num_seqs - at : kScoreSeqs;
        a.page_tables += static_cast<int64_t>(at) * num_kv_heads * max_pages;
        a.page_lens += at;
        a.q += static_cast<int64_t>(at) * num_q_heads * head_dim;
        a.block_tables += static_cast<int64_t>(at) * max_blocks_per_seq;
        a.seq_lens += at;
        cudaError_t e;
        switch (head_dim) {
            case 64: e = fp8 ? launch_select<64, true>(a, s) : launch_select<64, false>(a, s); break;
            case 128: e = fp8 ? launch_select<128, true>(a, s) : launch_select<128, false>(a, s); break;
            default: e = fp8 ? launch_select<256, true>(a, s) : launch_select<256, false>(a, s); break;
        }
        if (e != cudaSuccess) return api_cuda_fail(e, "page selection launch");
    }
    return PA_OK;
}
