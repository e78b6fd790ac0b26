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
//     E = (group + 16) 2^-24 S,  S >= sum_d |P_d max_d| + |N_d min_d| of any page
// (P and N are sums of `group` terms, a lane adds 16 products at most and five shuffles join
// the lanes: fewer than group + 16 ... roundings act on any product).  With T the f-th
// largest computed score, a page above T + 2E is among the f best and one below T - 2E is
// not; the band between is scored again in fp64 and ranked by (score, page).
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

// One warp per (sequence, page, kv head).  A row is CPR chunks of 16 bytes; the warp reads
// 32 / CPR rows per load instruction, every load in flight before the first comparison.
template <int HD, bool FP8>
__global__ void __launch_bounds__(256) bounds_kernel(const __grid_constant__ BoundsParams p) {
    constexpr int ROW = HD * (FP8 ? 1 : 2);
    constexpr int CPR = ROW / 16;
    constexpr int RPL = 32 / CPR;                 // rows per load
    constexpr int LOADS = kBlockSize / RPL;
    constexpr int W = FP8 ? 8 : 4;                // 16-bit pairs a lane holds
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t per_seq = static_cast<int64_t>(p.pages) * p.num_kv_heads;
    const int64_t b = unit / per_seq;
    if (b >= p.num_seqs) return;
    const int rest = static_cast<int>(unit - b * per_seq);
    const int kh = rest % p.num_kv_heads;
    int L = max(p.seq_lens[b], 0);
    const int first = p.first_tokens ? min(max(p.first_tokens[b], 0), L) : 0;
    const int cap = p.max_blocks * kBlockSize;
    bool bad = L > cap;
    L = min(L, cap);
    const int page = first / kBlockSize + rest / p.num_kv_heads;
    // the last unit of a sequence sees whether its pages go on past the launch's
    bad = bad || (L + kBlockSize - 1) / kBlockSize - first / kBlockSize > p.pages;
    if (bad && rest == 0 && lane == 0) atomicOr(p.status, kStatusBounds);
    const int rows = min(kBlockSize, L - page * kBlockSize);
    if (rows <= 0 || first >= L) return;
    const int id = p.block_tables[b * p.max_blocks + page];
    if (id < 0 || id >= p.num_blocks) {
        if (lane == 0) atomicOr(p.status, kStatusBounds);
        return;
    }
    const int c = lane % CPR, r0 = lane / CPR;
    const uint8_t *src = p.k_cache + id * p.b_block + kh * p.b_head + c * 16;
    uint4 raw[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {   // rows past the sequence repeat its last one
        const int r = min(i * RPL + r0, rows - 1);
        raw[i] = __ldg(reinterpret_cast<const uint4 *>(src + r * p.b_token));
    }
    uint32_t lo[W], hi[W];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
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
    if (lane >= CPR) return;
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

template <int HD>
cudaError_t launch_bounds(const BoundsParams &p, bool fp8, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(p.num_seqs) * p.pages * p.num_kv_heads;
    const unsigned grid = static_cast<unsigned>((units + 7) / 8);
    if (fp8) bounds_kernel<HD, true><<<grid, 256, 0, stream>>>(p);
    else bounds_kernel<HD, false><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

// ---- scores ---------------------------------------------------------------------------------

constexpr int kScorePages = 64;   // pages per CTA of the score kernel

struct SelectParams {
    int32_t *page_tables, *page_lens;
    const __nv_bfloat16 *q;
    const uint8_t *bounds;
    const int32_t *block_tables, *seq_lens;
    float *score;       // [B][nkv][max_blocks]
    float *span;        // [B][nkv][chunks]: largest S of a chunk's pages
    int32_t *band;      // [B][nkv][max_blocks]
    double *exact;      // [B][nkv][max_blocks]
    int64_t num_blocks;
    int num_seqs, nq, nkv, max_blocks, chunks, max_pages, sink, recent;
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

// A channel whose query weight is zero adds nothing, an infinite bound included.
template <typename T>
__device__ __forceinline__ T weighed(T w, T x) {
    return w == T(0) ? T(0) : w * x;
}

// Element d of a bounds row as a float.
template <bool FP8>
__device__ __forceinline__ float bound_value(const uint8_t *row, int d) {
    if constexpr (FP8) return e4m3x2_to_float2(row[d]).x;
    else return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[d]);
}

// Grid (chunk, kv head, sequence); a warp per page.  Lane l holds channels l * HD / 32 on of
// P and N.
template <int HD, bool FP8>
__global__ void __launch_bounds__(256) score_kernel(const __grid_constant__ SelectParams p) {
    constexpr int ROW = HD * (FP8 ? 1 : 2), D = HD / 32;
    __shared__ float span[8];
    const int b = blockIdx.z, kh = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int L = select_len(p, b, blockIdx.x == 0 && kh == 0 && threadIdx.x == 0);
    const int np = (L + kBlockSize - 1) / kBlockSize;
    const int first = blockIdx.x * kScorePages;
    if (np <= p.max_pages || first >= np) return;
    const int g = p.nq / p.nkv;
    float P[D], N[D];
    for (int d = 0; d < D; ++d) P[d] = N[d] = 0.f;
    for (int h = 0; h < g; ++h)
        for (int d = 0; d < D; ++d) {
            const float x = __bfloat162float(
                p.q[(static_cast<int64_t>(b) * p.nq + kh * g + h) * HD + lane * D + d]);
            P[d] += x >= 0.f || isnan(x) ? x : 0.f;
            N[d] += x < 0.f ? x : 0.f;
        }
    const int64_t row = static_cast<int64_t>(b) * p.nkv + kh;
    float most = 0.f;
    for (int i = first + warp; i < min(first + kScorePages, np); i += 8) {
        const int id = p.block_tables[static_cast<int64_t>(b) * p.max_blocks + i];
        float s = 0.f, a = 0.f;
        if (id < 0 || id >= p.num_blocks) {
            if (lane == 0) atomicOr(p.status, kStatusBounds);
            s = -INFINITY;
        } else {
            const uint8_t *lo = p.bounds + (static_cast<int64_t>(id) * p.nkv + kh) * 2 * ROW;
            for (int d = 0; d < D; ++d) {
                const float x = weighed(P[d], bound_value<FP8>(lo + ROW, lane * D + d));
                const float y = weighed(N[d], bound_value<FP8>(lo, lane * D + d));
                s += x + y;
                a += fabsf(x) + fabsf(y);
            }
            for (int o = 16; o; o >>= 1) {
                s += __shfl_xor_sync(kAll, s, o);
                a += __shfl_xor_sync(kAll, a, o);
            }
        }
        most = max_nan(most, a);
        if (lane == 0) p.score[row * p.max_blocks + i] = s;
    }
    if (lane == 0) span[warp] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) most = max_nan(most, span[w]);
        p.span[row * p.chunks + blockIdx.x] = most;
    }
}

// ---- selection ------------------------------------------------------------------------------

constexpr int kSelThreads = 1024;

// Order-preserving whole numbers of floating scores; a NaN is the largest.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (isnan(x)) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint64_t key_of(double x) {
    if (isnan(x)) return ~0ull;
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x == 0.0 ? 0.0 : x));
    return u >> 63 ? ~u : u | 1ull << 63;
}

// Exclusive prefix of x over the CTA, and the total.
__device__ __forceinline__ int block_scan(int x, int *warps, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) warps[warp] = v;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
        if (w < warp) before += warps[w];
        total += warps[w];
    }
    __syncthreads();
    return before + v - x;
}

// The f-th largest (f >= 1) of n keys, and how many exceed it: radix select, a byte a pass.
template <typename Key, typename Get>
__device__ __forceinline__ Key nth_largest(int n, int f, int *hist, Get get, int &greater) {
    __shared__ int pick[2];
    Key prefix = 0;
    int above = 0;
    for (int shift = static_cast<int>(sizeof(Key)) * 8 - 8; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kSelThreads) {
            const Key k = get(i);
            const bool in = shift + 8 >= static_cast<int>(sizeof(Key)) * 8 ||
                            (k >> (shift + 8)) == (prefix >> (shift + 8));
            if (in) atomicAdd(&hist[static_cast<int>(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int c = above, d = 255;
            while (d > 0 && c + hist[d] < f) c += hist[d--];
            pick[0] = d;
            pick[1] = c;
        }
        __syncthreads();
        prefix |= static_cast<Key>(pick[0]) << shift;
        above = pick[1];
        __syncthreads();
    }
    greater = above;
    return prefix;
}

// One CTA per (kv head, sequence).
template <int HD, bool FP8>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ SelectParams p) {
    constexpr int ROW = HD * (FP8 ? 1 : 2);
    __shared__ int hist[256];
    __shared__ int warps[kSelThreads / 32];
    __shared__ float span_sh;
    __shared__ double P[HD], N[HD];
    const int kh = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = select_len(p, b, false);
    const int np = (L + kBlockSize - 1) / kBlockSize;
    const int kept = min(np, p.max_pages);
    const int64_t row = static_cast<int64_t>(b) * p.nkv + kh;
    const int32_t *bt = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
    int32_t *out = p.page_tables + row * p.max_pages;
    if (kh == 0 && tid == 0) p.page_lens[b] = kept * kBlockSize - (np * kBlockSize - L);
    for (int i = kept + tid; i < p.max_pages; i += kSelThreads) out[i] = -1;
    if (np <= p.max_pages) {
        for (int i = tid; i < np; i += kSelThreads) out[i] = bt[i];
        return;
    }
    // f pages of [lo, hi) join the sinks and the newest ones
    const int lo = p.sink, hi = np - p.recent, f = p.max_pages - p.sink - p.recent;
    const float *score = p.score + row * p.max_blocks;
    int32_t *band = p.band + row * p.max_blocks;
    double *exact = p.exact + row * p.max_blocks;
    float above = INFINITY, below = INFINITY;   // sure winners exceed `above`, losers miss `below`
    int take = 0;                               // winners that come from the band
    uint64_t edge = 0;                          // the band's weakest winner ...
    int ties = 0;                               // ... and how many equal to it win
    bool all = true;                            // the whole band wins
    if (f > 0) {
        int greater;
        const uint32_t t =
            nth_largest<uint32_t>(hi - lo, f, hist, [&](int i) { return key_of(score[lo + i]); }, greater);
        if (tid == 0) {
            float s = 0.f;
            for (int i = 0; i < (np + kScorePages - 1) / kScorePages; ++i)
                s = max_nan(s, p.span[row * p.chunks + i]);
            span_sh = s;
        }
        __syncthreads();
        const float T = t == 0xffffffffu ? NAN
                                         : __uint_as_float(t & 0x80000000u ? t & 0x7fffffffu : ~t);
        const float E2 = 2.f * static_cast<float>(p.nq / p.nkv + 16) * 0x1p-24f * span_sh;
        above = T + E2;
        below = T - E2;
        // the band in page order
        int n_band = 0, n_above = 0;
        for (int base = lo; base < hi; base += kSelThreads) {
            const int i = base + tid;
            const float s = i < hi ? score[i] : 0.f;
            const bool win = i < hi && s > above, in = i < hi && !win && !(s < below);
            int total;
            const int at = block_scan((in ? 1 : 0) | (win ? 1 << 16 : 0), warps, total);
            if (in) band[n_band + (at & 0xffff)] = i;
            n_band += total & 0xffff;
            n_above += total >> 16;
        }
        take = f - n_above;
        all = take == n_band;
        if (!all) {
            const int g = p.nq / p.nkv;
            for (int d = tid; d < HD; d += kSelThreads) {
                double x = 0.0, y = 0.0;
                for (int h = 0; h < g; ++h) {
                    const float v = __bfloat162float(
                        p.q[(static_cast<int64_t>(b) * p.nq + kh * g + h) * HD + d]);
                    if (v < 0.f) y += v;
                    else x += v;
                }
                P[d] = x;
                N[d] = y;
            }
            __syncthreads();
            for (int i = warp; i < n_band; i += kSelThreads / 32) {
                const int id = bt[band[i]];
                double s = 0.0;
                if (id >= 0 && id < p.num_blocks) {
                    const uint8_t *r = p.bounds + (static_cast<int64_t>(id) * p.nkv + kh) * 2 * ROW;
                    for (int d = lane; d < HD; d += 32)
                        s += weighed<double>(P[d], bound_value<FP8>(r + ROW, d)) +
                             weighed<double>(N[d], bound_value<FP8>(r, d));
                    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
                } else {
                    s = -INFINITY;
                }
                if (lane == 0) exact[i] = s;
            }
            __syncthreads();
            int more;
            edge = nth_largest<uint64_t>(n_band, take, hist, [&](int i) { return key_of(exact[i]); }, more);
            ties = take - more;
        }
    }
    // the chosen pages in order
    int n_out = 0, n_band = 0, n_tie = 0;
    for (int base = 0; base < np; base += kSelThreads) {
        const int i = base + tid;
        const bool held = i < np && (i < lo || i >= hi);
        bool win = held, in = false;
        if (i < np && !held && f > 0) {
            const float s = score[i];
            win = s > above;
            in = !win && !(s < below);
        }
        int total;
        const int at = block_scan(in ? 1 : 0, warps, total);
        bool tie = false;
        if (in) {
            const uint64_t k = all ? 1 : key_of(exact[n_band + at]);
            win = all || k > edge;
            tie = !all && k == edge;
        }
        n_band += total;
        const int nth = block_scan(tie ? 1 : 0, warps, total);
        if (tie && n_tie + nth < ties) win = true;
        n_tie += total;
        const int to = block_scan(win ? 1 : 0, warps, total);
        if (win) out[n_out + to] = bt[i];
        n_out += total;
    }
}

template <int HD, bool FP8>
cudaError_t launch_select(const SelectParams &p, cudaStream_t stream) {
    if (p.max_blocks > p.max_pages) {
        score_kernel<HD, FP8><<<dim3(p.chunks, p.nkv, p.num_seqs), 256, 0, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    select_kernel<HD, FP8><<<dim3(p.nkv, p.num_seqs), kSelThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Offsets of the workspace's parts (scores, spans, band, exact scores) and its size.
size_t select_layout(int num_seqs, int nkv, int max_blocks, size_t off[4]) {
    const size_t rows = static_cast<size_t>(num_seqs > 0 ? num_seqs : 0) * (nkv > 0 ? nkv : 0);
    const size_t n = rows * (max_blocks > 0 ? max_blocks : 0);
    const size_t chunks = (static_cast<size_t>(max_blocks > 0 ? max_blocks : 0) + kScorePages - 1) / kScorePages;
    off[0] = 0;
    off[1] = off[0] + round256(n * 4);
    off[2] = off[1] + round256(rows * chunks * 4);
    off[3] = off[2] + round256(n * 4);
    return off[3] + round256(n * 8);
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
    int pages = (max_new_tokens + kBlockSize - 1) / kBlockSize;
    if (first_tokens) pages = (max_new_tokens + 2 * (kBlockSize - 1)) / kBlockSize;
    if (pages > max_blocks_per_seq) pages = max_blocks_per_seq;
    if (static_cast<int64_t>(num_seqs) * pages * num_kv_heads / 8 >= INT32_MAX)
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
    size_t off[4];
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
    if (max_pages <= 0 || max_pages > INT32_MAX / kBlockSize)
        return api_fail(PA_ERR_INVALID, "max_pages %d", max_pages);
    if (sink_pages < 0 || recent_pages < 1 || sink_pages > max_pages ||
        recent_pages > max_pages - sink_pages)
        return api_fail(PA_ERR_INVALID, "sink_pages %d and recent_pages %d (at least 1) in %d pages",
                        sink_pages, recent_pages, max_pages);
    if (num_seqs > 65535 || num_kv_heads > 65535)
        return api_fail(PA_ERR_UNSUPPORTED, "num_seqs %d, num_kv_heads %d: at most 65535", num_seqs,
                        num_kv_heads);
    if (num_seqs == 0) return PA_OK;
    if (!page_tables || !page_lens || !q || !bounds || !block_tables || !seq_lens)
        return api_fail(PA_ERR_INVALID, "null pointer argument");
    if (!aligned(q, 16) || !aligned(bounds, 16))
        return api_fail(PA_ERR_INVALID, "q and bounds must be 16-byte aligned");
    size_t off[4];
    const size_t need = select_layout(num_seqs, num_kv_heads, max_blocks_per_seq, off);
    if (workspace_bytes < need)
        return api_fail(PA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (!workspace || !aligned(workspace, 256))
        return api_fail(PA_ERR_WORKSPACE, "workspace must be non-null and 256-byte aligned");
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
    p.band = reinterpret_cast<int32_t *>(ws + off[2]);
    p.exact = reinterpret_cast<double *>(ws + off[3]);
    p.num_blocks = num_blocks;
    p.num_seqs = num_seqs;
    p.nq = num_q_heads;
    p.nkv = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.chunks = (max_blocks_per_seq + kScorePages - 1) / kScorePages;
    p.max_pages = max_pages;
    p.sink = sink_pages;
    p.recent = recent_pages;
    rc = api_status_ptr(&p.status);
    if (rc) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
    cudaError_t e;
    switch (head_dim) {
        case 64: e = fp8 ? launch_select<64, true>(p, s) : launch_select<64, false>(p, s); break;
        case 128: e = fp8 ? launch_select<128, true>(p, s) : launch_select<128, false>(p, s); break;
        default: e = fp8 ? launch_select<256, true>(p, s) : launch_select<256, false>(p, s); break;
    }
    if (e != cudaSuccess) return api_cuda_fail(e, "page selection launch");
    return PA_OK;
}
