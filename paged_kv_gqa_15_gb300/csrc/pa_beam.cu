// pa_beam.cu -- beam search's selection: per request the K best of all (beam, token) pairs by
//   score(b, t) = cum[b] + x[b][t] - log sum_t exp x[b][t].
//
// Two kernels.  The scan reads every live row once: a warp takes a run of 256-element chunks, keeps the
// run's maximum m and sum of exp(x - m), and writes each chunk's maximum (1 value for 256).  The pick, a CTA
// per request, joins the runs' sums into each beam's log-sum-exp, ranks the chunks by their maxima, and
// reads the K best chunks again: the K best elements lie in them (an element outside is outranked by the K
// maxima of the chunks before its own).
//
// Order.  Within a beam the order of scores is that of the logits, across beams it needs the sums, so a
// score is kept as an unevaluated sum of two fp32 (48 bits: differences and sums with their rounding errors):
// two logits next to each other in fp32 stay apart behind an offset of any usual size.  Equal scores go to
// the lower beam, then the lower token.  The sums come from ex2.approx (2^-22 relative) in
// compensated fp32, so that cum - logsumexp is known to better than 2^-20, and equal rows get equal sums:
// chunks and lanes are counted from the row's start.
//
// Bound by reading the logits once (the chunk maxima add 1/128 of bf16 logits).
#include <cmath>
#include <cstring>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kChunk = 256;                  // logits whose maximum is kept
constexpr int kScanThreads = 256;
constexpr int kPickThreads = 1024;
constexpr int kAhead = 4;                    // chunks of a warp's run that are on their way at once
constexpr int kMostCandidates = 1024;        // ranked by counting; more of them take the slow way

struct BeamParams {
    float *scores;
    int32_t *beams, *tokens;
    const void *logits;
    const float *cum;
    const uint8_t *finished;                 // or null
    float *chunk_max;                        // [rows][chunks]
    float2 *runs;                            // [rows][num_runs]: maximum, sum of exp(x - maximum)
    int64_t row_stride;
    int num_requests, num_beams, vocab, num_out, end_token;
    int chunks, run_chunks, num_runs;
    int *status;
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}

// s + e plus x, the rounding error of the sum gathered in e.
__device__ __forceinline__ void add_compensated(float &s, float &e, float x) {
    const float t = s + x, z = t - s;
    e += (s - (t - z)) + (x - z);
    s = t;
}

// Whether a row's logits are read: not those of a beam that is finished or out of the search.
__device__ __forceinline__ bool row_is_read(const BeamParams &p, int64_t row) {
    return p.cum[row] > -INFINITY && !(p.finished && p.finished[row]);
}

// The eight logits of a lane in one chunk: adjacent ones in vectors where rows start at 16 bytes, else
// every 32nd; past the row's end -inf.
template <typename T, bool VECTORS>
__device__ __forceinline__ void load8(const T *row, int at, int vocab, int lane, float (&x)[8]) {
    constexpr bool kWide = sizeof(T) == 4;
    if (VECTORS && at + kChunk <= vocab) {
        if (kWide) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(row + at) + lane + 32 * i);
                x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
            }
        } else {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(row + at) + lane);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = at + (!VECTORS ? lane + 32 * i : kWide ? 4 * lane + i % 4 + i / 4 * 128 : 8 * lane + i);
        x[i] = c < vocab ? static_cast<float>(row[c]) : -INFINITY;
    }
}

template <typename T, bool VECTORS>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const __grid_constant__ BeamParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kScanThreads / 32) + threadIdx.x / 32;
    const int64_t row = w / p.num_runs;
    const int run = static_cast<int>(w - row * p.num_runs);
    if (row >= static_cast<int64_t>(p.num_requests) * p.num_beams || !row_is_read(p, row)) return;
    const T *logits = static_cast<const T *>(p.logits) + row * p.row_stride;
    float *best = p.chunk_max + row * p.chunks;
    const int c_end = min(p.chunks, (run + 1) * p.run_chunks);
    float m = -INFINITY, s = 0.f, e = 0.f;
    for (int c0 = run * p.run_chunks; c0 < c_end; c0 += kAhead) {
        float x[kAhead][8];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            if (c0 + a < c_end) load8<T, VECTORS>(logits, (c0 + a) * kChunk, p.vocab, lane, x[a]);
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            if (c0 + a >= c_end) break;
            float top = x[a][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, x[a][i]);
            top = warp_max(top);
            if (lane == 0) best[c0 + a] = top;
            if (top > m) {                       // the same in every lane
                const float f = exp2_approx((m - top) * kLog2e);
                s *= f, e *= f;
                m = top;
            }
            const float base = m == -INFINITY ? 0.f : m;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = exp2_approx((x[a][i] - base) * kLog2e);
            add_compensated(s, e, ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7])));
        }
    }
    s += e;
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) p.runs[row * p.num_runs + run] = make_float2(m, s);
}

// ---- the pick ---------------------------------------------------------------------------

// A score and where it stands: the greater key first, then the lower place.  key 0: nothing.
struct Ranked {
    uint64_t key;
    uint32_t place;
};

__device__ __forceinline__ bool before(const Ranked &a, const Ranked &b) {
    return a.key > b.key || (a.key == b.key && a.place < b.place);
}

// Bits of x in an order of unsigned numbers; -0 as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// What a beam's logits have added to them to become scores: x - top + (hi + lo).
struct Offset {
    float top, hi, lo;                       // the largest logit; cum - log sum exp(x - top) as two fp32
};

// The score of logit x as a key of two fp32; 0 where it is -inf (or not a number).
__device__ __forceinline__ uint64_t key_of(float x, const Offset &o) {
    const float d = x - o.top, y = d - x;
    const float s = d + o.hi, z = s - d;
    const float e = (d - (s - z)) + (o.hi - z) + ((x - (d - y)) - (o.top + y) + o.lo);
    const float top = s + e, rest = e - (top - s);
    if (!(top > -INFINITY)) return 0;
    return static_cast<uint64_t>(ordered(top)) << 32 | ordered(rest);
}

__device__ __forceinline__ float score_of(uint64_t key) {
    const uint32_t b = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}

__device__ __forceinline__ Ranked shuffle_down_best(Ranked r, int d) {
    Ranked o;
    o.key = __shfl_xor_sync(0xffffffffu, r.key, d);
    o.place = __shfl_xor_sync(0xffffffffu, r.place, d);
    return before(o, r) ? o : r;
}

struct PickSpace {
    Ranked found[kMostCandidates];
    Ranked groups[kPickThreads / 8];
    Ranked bar;                              // a candidate is not behind it
    Ranked chosen[PA_MAX_BEAM_OUT];
    int count;
    Offset offset[PA_MAX_BEAMS];
    int kind[PA_MAX_BEAMS];                  // 0: out, 1: live, 2: finished
};

// The `most` first of item(0) .. item(n - 1), in order, into sp.chosen; returns how many there are (items
// of key 0 do not count).  Called by the whole CTA; places are all different.
//
// Each of 32 to 128 groups of threads finds its first item; the most-th of these is a bar that `most`
// items pass, so that only items that pass it can be among the first.  They are few, and ranked by
// counting.  Where too many pass (the items of few groups are before all others), the first are taken one
// by one instead.
template <typename Item>
__device__ int pick(PickSpace &sp, int n, int most, const Item &item) {
    const int tid = threadIdx.x;
    // groups at least twice `most`, so that the bar is not pulled down by an unlucky group
    const int lanes = most <= 16 ? 32 : most <= 32 ? 16 : 8;
    const int groups = kPickThreads / lanes;
    Ranked first = {0, 0xffffffffu};
    for (int i = tid; i < n; i += kPickThreads) {
        const Ranked r = item(i);
        if (before(r, first)) first = r;
    }
    for (int d = 1; d < lanes; d <<= 1) first = shuffle_down_best(first, d);
    if (tid % lanes == 0) sp.groups[tid / lanes] = first;
    if (tid == 0) sp.count = 0, sp.bar = {1, 0xffffffffu};
    __syncthreads();
    if (tid < groups) {
        const Ranked mine = sp.groups[tid];
        int rank = 0;
        for (int g = 0; g < groups; ++g) rank += before(sp.groups[g], mine);
        if (mine.key && rank == most - 1) sp.bar = mine;
    }
    __syncthreads();
    const Ranked bar = sp.bar;
    for (int i = tid; i < n; i += kPickThreads) {
        const Ranked r = item(i);
        if (r.key && !before(bar, r)) {
            const int at = atomicAdd(&sp.count, 1);
            if (at < kMostCandidates) sp.found[at] = r;
        }
    }
    __syncthreads();
    const int count = sp.count;
    if (count <= kMostCandidates) {
        for (int i = tid; i < count; i += kPickThreads) {
            const Ranked mine = sp.found[i];
            int rank = 0;
            for (int j = 0; j < count; ++j) rank += before(sp.found[j], mine);
            if (rank < most) sp.chosen[rank] = mine;
        }
        __syncthreads();
        return min(count, most);
    }
    Ranked last = {~0ull, 0};
    for (int k = 0; k < most; ++k) {
        Ranked next = {0, 0xffffffffu};
        for (int i = tid; i < n; i += kPickThreads) {
            const Ranked r = item(i);
            if (before(last, r) && before(r, next)) next = r;
        }
        for (int d = 1; d < 32; d <<= 1) next = shuffle_down_best(next, d);
        if (tid % 32 == 0) sp.groups[tid / 32] = next;
        __syncthreads();
        if (tid < 32) {
            next = sp.groups[tid];
            for (int d = 1; d < 32; d <<= 1) next = shuffle_down_best(next, d);
            if (tid == 0) sp.chosen[k] = next;
        }
        __syncthreads();
        last = sp.chosen[k];
        if (!last.key) return k;
    }
    return most;
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const __grid_constant__ BeamParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ PickSpace sp;
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.num_beams;
    // cum - logsumexp of every beam
    for (int b = tid / 32; b < p.num_beams; b += kPickThreads / 32) {
        const float cum = p.cum[row0 + b];
        const bool finished = p.finished && p.finished[row0 + b];
        int kind = cum == -INFINITY ? 0 : finished ? 2 : 1;
        Offset offset = {0.f, cum, 0.f};
        bool bad = !(cum < INFINITY);
        if (kind == 1 && !bad) {
            const float2 *runs = p.runs + (row0 + b) * p.num_runs;
            float m = -INFINITY;
            for (int i = lane; i < p.num_runs; i += 32) m = fmaxf(m, runs[i].x);
            m = warp_max(m);
            float s = 0.f, e = 0.f;
            for (int i = lane; i < p.num_runs; i += 32) {
                const float2 r = runs[i];
                // an empty run (its maximum -inf) has a sum of 0, or NaN
                add_compensated(s, e, r.y * (r.x == m ? 1.f : exp2_approx((r.x - m) * kLog2e)));
            }
            s += e;
#pragma unroll
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            bad = !(m < INFINITY) || s != s;
            if (m == -INFINITY) kind = 0;      // every token is ruled out
            // log of s = 2^n f, f within [0.7, 1.5): the large part exactly, the small one in fp32
            int n;
            float f = frexpf(s, &n);
            if (f < 0.70710678f) f *= 2.f, n -= 1;
            const double off = cum - n * 0.6931471805599453 - static_cast<double>(logf(f));
            const float hi = static_cast<float>(off);
            offset = {m, hi, static_cast<float>(off - hi)};
        }
        if (bad) kind = 0;
        if (lane == 0) {
            if (bad) atomicOr(p.status, kStatusInvalid);
            sp.kind[b] = kind;
            sp.offset[b] = offset;
        }
    }
    __syncthreads();
    const int chunks = p.chunks;
    const float *best = p.chunk_max + row0 * chunks;
    const int kept = pick(sp, p.num_beams * chunks, p.num_out, [&](int i) -> Ranked {
        const int b = i / chunks;
        const int kind = sp.kind[b];
        if (kind == 1) return {key_of(best[i], sp.offset[b]), static_cast<uint32_t>(i)};
        if (kind == 2 && i == b * chunks) return {key_of(0.f, sp.offset[b]), static_cast<uint32_t>(i)};
        return {0, static_cast<uint32_t>(i)};
    });
    __shared__ uint32_t from[PA_MAX_BEAM_OUT];
    if (tid < kept) from[tid] = sp.chosen[tid].place;
    __syncthreads();
    const T *logits = static_cast<const T *>(p.logits) + row0 * p.row_stride;
    const int got = pick(sp, kept * kChunk, p.num_out, [&](int i) -> Ranked {
        const int c = static_cast<int>(from[i / kChunk]);
        const int b = c / chunks;
        const int token = (c - b * chunks) * kChunk + i % kChunk;
        if (sp.kind[b] == 2) {
            // one candidate of the whole beam
            if (i % kChunk) return {0, 0xffffffffu};
            return {key_of(0.f, sp.offset[b]), static_cast<uint32_t>(b) * p.vocab + p.end_token};
        }
        if (token >= p.vocab) return {0, 0xffffffffu};
        const float x = static_cast<float>(logits[b * p.row_stride + token]);
        return {key_of(x, sp.offset[b]), static_cast<uint32_t>(b) * p.vocab + token};
    });
    if (tid < p.num_out) {
        const int64_t at = static_cast<int64_t>(blockIdx.x) * p.num_out + tid;
        const bool real = tid < got;
        const uint32_t place = real ? sp.chosen[tid].place : 0;
        p.scores[at] = real ? score_of(sp.chosen[tid].key) : -INFINITY;
        p.beams[at] = real ? static_cast<int>(place / p.vocab) : -1;
        p.tokens[at] = real ? static_cast<int>(place % p.vocab) : -1;
    }
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int64_t chunks_of(int vocab) { return (static_cast<int64_t>(vocab) + kChunk - 1) / kChunk; }

template <typename T>
cudaError_t launch_select(const BeamParams &p, cudaStream_t stream) {
    const int64_t warps = static_cast<int64_t>(p.num_requests) * p.num_beams * p.num_runs;
    const dim3 grid(static_cast<unsigned>((warps + kScanThreads / 32 - 1) / (kScanThreads / 32)));
    const bool vectors = (reinterpret_cast<uintptr_t>(p.logits) & 15u) == 0 && p.row_stride % (16 / sizeof(T)) == 0;
    const cudaError_t e = vectors ? launch_after(beam_scan_kernel<T, true>, grid, kScanThreads, p, stream)
                                  : launch_after(beam_scan_kernel<T, false>, grid, kScanThreads, p, stream);
    if (e != cudaSuccess) return e;
    return launch_after(beam_pick_kernel<T>, dim3(static_cast<unsigned>(p.num_requests)), kPickThreads, p, stream);
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_beam_select_workspace_size(int num_requests, int num_beams, int vocab) {
    using namespace pa;
    if (num_requests <= 0 || num_beams <= 0 || vocab <= 0) return 0;
    const size_t n = static_cast<size_t>(num_requests) * num_beams * static_cast<size_t>(chunks_of(vocab));
    return round256(n * sizeof(float)) + round256(n * sizeof(float2));
}

extern "C" int pa_beam_select(float *scores, int32_t *beams, int32_t *tokens, const void *logits,
                              const float *cum_scores, const uint8_t *finished, int end_token, int num_requests,
                              int num_beams, int vocab, int num_out, int64_t stride_row, int logits_dtype,
                              void *workspace, size_t workspace_bytes, void *stream) {
    using namespace pa;
    if (num_requests < 0) return api_fail(PA_ERR_INVALID, "num_requests %d", num_requests);
    if (num_beams <= 0 || vocab <= 0 || num_out <= 0)
        return api_fail(PA_ERR_INVALID, "num_beams %d, vocab %d, num_out %d must be positive", num_beams, vocab, num_out);
    if (num_beams > PA_MAX_BEAMS || num_out > PA_MAX_BEAM_OUT || vocab > PA_MAX_BEAM_VOCAB)
        return api_fail(PA_ERR_UNSUPPORTED, "num_beams %d > %d, num_out %d > %d or vocab %d > %d", num_beams, PA_MAX_BEAMS,
                        num_out, PA_MAX_BEAM_OUT, vocab, PA_MAX_BEAM_VOCAB);
    if (logits_dtype != PA_LOGITS_F32 && logits_dtype != PA_LOGITS_BF16)
        return api_fail(PA_ERR_UNSUPPORTED, "logits_dtype %d", logits_dtype);
    if (stride_row < vocab && num_requests * static_cast<int64_t>(num_beams) > 1)
        return api_fail(PA_ERR_INVALID, "stride_row %lld < vocab %d", static_cast<long long>(stride_row), vocab);
    if (stride_row > (INT64_C(1) << 40))
        return api_fail(PA_ERR_UNSUPPORTED, "stride_row %lld", static_cast<long long>(stride_row));
    if (finished && (end_token < 0 || end_token >= vocab))
        return api_fail(PA_ERR_INVALID, "end_token %d not in [0, %d)", end_token, vocab);
    if (num_requests == 0) return PA_OK;
    if (!scores || !beams || !tokens || !logits || !cum_scores)
        return api_fail(PA_ERR_INVALID, "null pointer argument");
    const size_t elem = logits_dtype == PA_LOGITS_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(logits) % elem) return api_fail(PA_ERR_INVALID, "logits are not aligned to their type");
    const int64_t outs = static_cast<int64_t>(num_requests) * num_out;
    const int64_t rows = static_cast<int64_t>(num_requests) * num_beams;
    const int32_t *written[3] = {reinterpret_cast<int32_t *>(scores), beams, tokens};
    for (int i = 0; i < 3; ++i) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(written[i]), end = at + outs * 4;
        auto over = [&](const void *x, int64_t bytes) {
            const uintptr_t b = reinterpret_cast<uintptr_t>(x);
            return at < b + bytes && b < end;
        };
        if (over(written[(i + 1) % 3], outs * 4) || over(cum_scores, rows * 4) || (finished && over(finished, rows)) ||
            over(logits, ((rows - 1) * stride_row + vocab) * elem))
            return api_fail(PA_ERR_INVALID, "scores, beams and tokens must overlap neither what the call reads nor one another");
    }
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < pa_beam_select_workspace_size(num_requests, num_beams, vocab))
        return api_fail(PA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed, 256-byte aligned", workspace_bytes,
                        pa_beam_select_workspace_size(num_requests, num_beams, vocab));
    BeamParams p;
    std::memset(&p, 0, sizeof p);
    p.scores = scores;
    p.beams = beams;
    p.tokens = tokens;
    p.logits = logits;
    p.cum = cum_scores;
    p.finished = finished;
    p.row_stride = stride_row;
    p.num_requests = num_requests;
    p.num_beams = num_beams;
    p.vocab = vocab;
    p.num_out = num_out;
    p.end_token = end_token;
    p.chunks = static_cast<int>(chunks_of(vocab));
    // runs: about the 64 warps that an SM holds, for each SM; short ones where there is little to read
    const int64_t share = (rows * p.chunks + 152 * 64 - 1) / (152 * 64);
    p.run_chunks = static_cast<int>(share < p.chunks ? share : p.chunks);
    p.num_runs = (p.chunks + p.run_chunks - 1) / p.run_chunks;
    const int64_t scan_ctas = (rows * p.num_runs + kScanThreads / 32 - 1) / (kScanThreads / 32);
    if (scan_ctas > INT32_MAX) return api_fail(PA_ERR_UNSUPPORTED, "%lld rows", static_cast<long long>(rows));
    p.chunk_max = static_cast<float *>(workspace);
    p.runs = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) +
                                        round256(static_cast<size_t>(rows) * p.chunks * sizeof(float)));
    int rc = api_status_ptr(&p.status);
    if (rc) return rc;
    const cudaError_t e = logits_dtype == PA_LOGITS_F32
                              ? launch_select<float>(p, static_cast<cudaStream_t>(stream))
                              : launch_select<__nv_bfloat16>(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : api_cuda_fail(e, "beam_select launch");
}
