// pa_beam.cu -- beam search's selection: per request the K best of all (beam, token) pairs by
//   score(b, t) = cum[b] + x[b][t] - log sum_t exp x[b][t].
//
// Two kernels.  The scan reads every live row once: a warp takes a share of its 256-element chunks (a
// run), keeps their sum of exp(x - m), m close to their maximum, and writes each chunk's maximum (1 value for 256).  The
// pick, a CTA per request, joins the runs' sums into each beam's log-sum-exp, finds the chunks that can be among the K
// best by their maxima, and reads those again: the K best elements lie in them (an element outside is
// outranked by the K maxima of the chunks before its own).
//
// Order.  Within a beam the order of scores is that of the logits, across beams it needs the sums, so a
// score is kept as an unevaluated sum of two fp32 (48 bits: differences and sums with their rounding errors):
// two logits next to each other in fp32 stay apart behind an offset of any usual size.  Equal scores go to
// the lower beam, then the lower token.  The sums come from ex2.approx (2^-22 relative) in compensated fp32.
// An exponent (x - m) log2 e is rounded twice, and what a run, or the join of the runs, counts from another m is
// multiplied once more: each step is off by 1.3 x 2^-20 over a distance of 8 and 1.7 over 12, ex2 included.  At most
// three steps behind an element's own matter (what lies e^-24 below is nothing even of 2^24 logits); they cost 5 x
// 2^-20 in all, the additions and the logarithm 1.2: cum - logsumexp is known to 2^-17.  Equal rows get equal sums:
// chunks and lanes are counted from the row's start.
//
// The scan is bound by reading the logits once (the chunk maxima add 1/128 of bf16 logits): 64 requests x 8
// beams x 128000 bf16, 131 MB, in about 21 us, 93 % of the copy rate; the pick behind it is a chain of 6 us.
// The call takes 27 us; captured, 4 beams x 32000 fp32 6.3, 12 x 5 x 50001 fp32 8.3.  Few requests that are not being
// captured take one launch instead of the two.
#include <cmath>
#include <cstring>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kChunk = 256;                  // logits whose maximum is kept
constexpr float kAbove = 8.f;                // what a run's largest logit may lie above the one it counts from
constexpr int kScanThreads = 256;
constexpr int kScanWarps = 152 * 32;         // that are on the GPU at a time
constexpr int kPickThreads = 1024;
constexpr int kCluster = 8;                  // CTAs of beam_small_kernel that share a request
constexpr int kSmallRequests = 15;
constexpr int kGroups = 2 * PA_MAX_BEAM_OUT; // of its threads at most, whose best scores make a bar
constexpr int kMostCandidates = 1024;        // ranked by counting; more of them take the slow way

struct BeamParams {
    float *scores;
    int32_t *beams, *tokens;
    const void *logits;
    const float *cum;
    const uint8_t *finished;                 // or null
    float *chunk_max;                        // [rows][chunks]
    float2 *runs;                            // [rows][num_runs]: a logit m within kAbove of the maximum, sum of exp(x - m)
    int64_t row_stride;
    int num_requests, num_beams, vocab, num_out, end_token;
    int chunks, num_runs;
    uint64_t per_chunk;                      // 2^40 / chunks, rounded up: i * per_chunk >> 40 is i / chunks
    int *status;
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The warp's largest x that is a number.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// s + e plus x, the rounding error of the sum gathered in e.
__device__ __forceinline__ void add_compensated(float &s, float &e, float x) {
    const float t = s + x, z = t - s;
    e += (s - (t - z)) + (x - z);
    s = t;
}

// Two fp32 in one register pair, for the instructions that work on both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float2 split(uint64_t a) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
    return d;
}

// Whether a row's logits are read: not those of a beam that is finished or out of the search.
__device__ __forceinline__ bool row_is_read(const BeamParams &p, int64_t row) {
    return p.cum[row] > -INFINITY && !(p.finished && p.finished[row]);
}

// 16 bytes that are read once.  (Volatile: the first of them are asked for before the warp knows that it
// has to read them.)
__device__ __forceinline__ uint4 stream(const uint4 *from) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(from));
    return v;
}

// A lane's eight logits of one chunk: adjacent ones where all rows start at 16 bytes, else pairs of bf16 or
// single fp32 values a warp's width apart; -inf past the row's end.
template <typename T>
struct Eight;

template <>
struct Eight<__nv_bfloat16> {
    static constexpr int kAhead = 4;             // chunks that a warp reads at once: 64 bytes a lane
    uint4 v;
    uint32_t last;                               // of a row that starts between two words
    // the chunk that starts at `chunk`, of which `left` logits are in the row
    template <bool VECTORS, bool WHOLE>
    __device__ __forceinline__ void load(const __nv_bfloat16 *chunk, int left, int lane) {
        if constexpr (VECTORS && WHOLE) {
            v = stream(reinterpret_cast<const uint4 *>(chunk) + lane);
        } else if constexpr (WHOLE) {
            // whole words; where the chunk starts in the middle of one, lane l has elements 2 l - 1 and 2 l of every
            // 64, and the chunk's last one is fetched apart
            const uint32_t *words = reinterpret_cast<const uint32_t *>(reinterpret_cast<uintptr_t>(chunk) & ~uintptr_t{3}) + lane;
            v = make_uint4(__ldg(words), __ldg(words + 32), __ldg(words + 64), __ldg(words + 96));
            if (lane == 0) last = __ldg(reinterpret_cast<const uint16_t *>(chunk) + kChunk - 1);
        } else {
            const uint16_t *bits = reinterpret_cast<const uint16_t *>(chunk);
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = VECTORS ? 8 * lane + i : 2 * lane + i % 2 + i / 2 * 64;
                w[i] = c < left ? __ldg(bits + c) : 0xff80u;
            }
            v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        }
    }
    // of a whole chunk that starts in the middle of a word: elements 2 l and 2 l + 1, when they are there
    __device__ __forceinline__ void settle(int lane) {
        const uint32_t w[5] = {v.x, v.y, v.z, v.w, last};
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            u[j] = __funnelshift_r(w[j], __shfl_sync(0xffffffffu, lane ? w[j] : w[j + 1], (lane + 1) & 31), 16);
        v = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ __forceinline__ float top() const {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ __forceinline__ uint64_t two(int i) const {
        const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
        return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};

template <>
struct Eight<float> {
    static constexpr int kAhead = 2;
    float4 v[2];
    template <bool VECTORS, bool WHOLE>
    __device__ __forceinline__ void load(const float *chunk, int left, int lane) {
        float x[8];
        if constexpr (VECTORS && WHOLE) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 w = stream(reinterpret_cast<const uint4 *>(chunk) + lane + 32 * i);
                x[4 * i] = __uint_as_float(w.x), x[4 * i + 1] = __uint_as_float(w.y);
                x[4 * i + 2] = __uint_as_float(w.z), x[4 * i + 3] = __uint_as_float(w.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = VECTORS ? 4 * lane + i % 4 + i / 4 * 128 : lane + 32 * i;
                x[i] = WHOLE || c < left ? __ldg(chunk + c) : -INFINITY;
            }
        }
        v[0] = make_float4(x[0], x[1], x[2], x[3]);
        v[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
    __device__ __forceinline__ void settle(int) {}
    __device__ __forceinline__ float top() const {
        return fmaxf(fmaxf(fmaxf(v[0].x, v[0].y), fmaxf(v[0].z, v[0].w)),
                     fmaxf(fmaxf(v[1].x, v[1].y), fmaxf(v[1].z, v[1].w)));
    }
    __device__ __forceinline__ uint64_t two(int i) const {
        const float4 &q = v[i / 2];
        return i % 2 ? pair(q.z, q.w) : pair(q.x, q.y);
    }
};

// A row's groups of chunks go to num_runs warps in turn, so that they read it side by side; a warp's next
// group is on its way while it works on one.  The logit m that exponents are counted from is the warp's, so that a
// group needs one comparison and, seldom, one rescaling.  It is no more than kAbove below the largest logit so
// far: every rescaling costs some 2^-20, and where m followed each new maximum a long row that rises from end to
// end gathered hundreds of them.  By steps of kAbove, what has been rescaled three times is e^-24 of the sum.
template <typename T, bool VECTORS>
__device__ __forceinline__ void scan_run(const BeamParams &p, int row, int run) {
    constexpr int kAhead = Eight<T>::kAhead;
    const int lane = threadIdx.x & 31;
    const T *logits = static_cast<const T *>(p.logits) + row * p.row_stride;
    float *best = p.chunk_max + static_cast<int64_t>(row) * p.chunks;
    // whether the row, and so each of its chunks, starts in the middle of a word
    const bool between = !VECTORS && sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(logits) & 2u);
    // groups of whole chunks, shared out in turn; what is left after them is the next warp's
    const int whole = p.vocab / kChunk, groups = whole / kAhead;
    float m = -INFINITY, s = 0.f, e = 0.f;
    auto rise = [&](float top) {                 // to a larger logit
        const float f = exp2_approx((m - top) * kLog2e);
        s *= f, e *= f;
        m = top;
    };
    auto sum_of = [&](const Eight<T> &x, uint64_t low) {
        const uint64_t scale = pair(kLog2e, kLog2e);
        uint64_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 z = split(mul2(add2(x.two(i), low), scale));
            y[i] = pair(exp2_approx(z.x), exp2_approx(z.y));
        }
        return add2(add2(y[0], y[1]), add2(y[2], y[3]));
    };
    const T *from = logits + run * (kAhead * kChunk);
    const int step = p.num_runs * (kAhead * kChunk);
    Eight<T> x[kAhead], next[kAhead];
    auto fetch = [&](Eight<T> (&to)[kAhead]) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) to[a].template load<VECTORS, true>(from + a * kChunk, kChunk, lane);
        from += step;
    };
    if (run < groups) fetch(x);                  // beside the row's cum and flag
    if (!row_is_read(p, row)) return;
#pragma unroll 2
    for (int g = run; g < groups; g += p.num_runs) {
        if (g + p.num_runs < groups) fetch(next);
        if (between)
#pragma unroll
            for (int a = 0; a < kAhead; ++a) x[a].settle(lane);
        float mine = -INFINITY, top = m;
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const float t = warp_max(x[a].top());
            top = fmaxf(top, t);
            if (lane == a) mine = t;
        }
        if (lane < kAhead) best[g * kAhead + lane] = mine;
        if (top > m + kAbove) rise(top);
        const float low = m == -INFINITY ? 0.f : -m;
        uint64_t sum[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) sum[a] = sum_of(x[a], pair(low, low));
#pragma unroll
        for (int d = 1; d < kAhead; d *= 2)
#pragma unroll
            for (int a = 0; a + d < kAhead; a += 2 * d) sum[a] = add2(sum[a], sum[a + d]);
        const float2 both = split(sum[0]);
        add_compensated(s, e, both.x + both.y);
#pragma unroll
        for (int a = 0; a < kAhead; ++a) x[a] = next[a];
    }
    for (int c = run == groups % p.num_runs ? groups * kAhead : p.chunks; c < p.chunks; ++c) {
        const T *chunk = logits + static_cast<int64_t>(c) * kChunk;
        if (c < whole) {
            x[0].template load<VECTORS, true>(chunk, kChunk, lane);
            if (between) x[0].settle(lane);
        } else {
            x[0].template load<VECTORS, false>(chunk, p.vocab - c * kChunk, lane);
        }
        const float top = warp_max(x[0].top());
        if (lane == 0) best[c] = top;
        if (top > m + kAbove) rise(top);
        const float low = m == -INFINITY ? 0.f : -m;
        const float2 both = split(sum_of(x[0], pair(low, low)));
        add_compensated(s, e, both.x + both.y);
    }
    s += e;
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) p.runs[static_cast<int64_t>(row) * p.num_runs + run] = make_float2(m, s);
}

template <typename T, bool VECTORS>
__global__ void __launch_bounds__(kScanThreads, 4) beam_scan_kernel(const __grid_constant__ BeamParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int w = blockIdx.x * (kScanThreads / 32) + threadIdx.x / 32;
    const int row = w / p.num_runs;
    if (row < p.num_requests * p.num_beams) scan_run<T, VECTORS>(p, row, w - row * p.num_runs);
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
    float top, hi, lo;                       // a logit near the largest; cum - log sum exp(x - top) as two fp32
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

__device__ __forceinline__ uint32_t head_of(uint64_t key) { return static_cast<uint32_t>(key >> 32); }

__device__ __forceinline__ float float_of(uint32_t ordered_bits) {
    return __uint_as_float(ordered_bits & 0x80000000u ? ordered_bits & 0x7fffffffu : ~ordered_bits);
}

enum { kOut = 0, kLive = 1, kFinished = 2 };

struct PickSpace {
    uint64_t key[2][kMostCandidates];        // the candidates among the chunks, among the elements
    uint32_t place[2][kMostCandidates];
    int count[2];
    __align__(16) uint32_t groups[kGroups];
    uint32_t bar;
    uint32_t reach;                          // largest |hi| of the beams, as bits
    int live;                                // beams whose chunks take part
    uint64_t chosen_key[PA_MAX_BEAM_OUT];
    uint32_t chosen[PA_MAX_BEAM_OUT], from[PA_MAX_BEAM_OUT];   // the first pairs, the chunks that hold them
    Ranked warps[kPickThreads / 32];
    Offset offset[PA_MAX_BEAMS];
    float2 shift[PA_MAX_BEAMS];              // of a live beam: (top, hi); of the others (0, -inf)
    int kind[PA_MAX_BEAMS];
};

__device__ __forceinline__ void note(PickSpace &sp, int stage, uint64_t key, uint32_t place) {
    const int at = atomicAdd(&sp.count[stage], 1);
    if (at < kMostCandidates) sp.key[stage][at] = key, sp.place[stage][at] = place;
}

// The `most` first of the candidates into sp.chosen, in order; returns how many there are.  Each warp
// counts who is before its candidates.  Where there were more candidates than room, the first of item(0)
// .. item(n - 1) are taken one by one instead (items of key 0 are none).
template <typename Item>
__device__ int rank(PickSpace &sp, int stage, int n, int most, const Item &item) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int count = sp.count[stage];
    if (count <= kMostCandidates) {
        for (int i = warp; i < count; i += kPickThreads / 32) {
            const Ranked mine = {sp.key[stage][i], sp.place[stage][i]};
            int r = 0;
            for (int j = lane; j < count; j += 32) r += before({sp.key[stage][j], sp.place[stage][j]}, mine);
            r = __reduce_add_sync(0xffffffffu, r);
            if (lane == 0 && r < most) sp.chosen_key[r] = mine.key, sp.chosen[r] = mine.place;
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
        for (int round = 0; round < 2; ++round) {
            for (int d = 1; d < 32; d <<= 1) {
                Ranked o;
                o.key = __shfl_xor_sync(0xffffffffu, next.key, d);
                o.place = __shfl_xor_sync(0xffffffffu, next.place, d);
                if (before(o, next)) next = o;
            }
            if (round) break;
            if (lane == 0) sp.warps[warp] = next;
            __syncthreads();
            next = sp.warps[lane];
        }
        __syncthreads();                     // before the next round's warps are written
        last = next;                         // the same in all threads
        if (!last.key) return k;
        if (tid == 0) sp.chosen_key[k] = last.key, sp.chosen[k] = last.place;
    }
    __syncthreads();
    return most;
}

// The most-th largest of the groups' values into sp.bar (0 if there are not so many).  By the whole CTA.
__device__ __noinline__ void raise_bar(PickSpace &sp, int groups, int most) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid < groups) {
        const uint32_t mine = sp.groups[tid];
        int r = 0;
        for (int g = 0; g < groups; g += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(sp.groups + g);
            r += (v.x > mine || (v.x == mine && g < tid)) + (v.y > mine || (v.y == mine && g + 1 < tid)) +
                 (v.z > mine || (v.z == mine && g + 2 < tid)) + (v.w > mine || (v.w == mine && g + 3 < tid));
        }
        if (r == most - 1) sp.bar = mine;
    }
    __syncthreads();
}

// cum - logsumexp of one beam, by a warp.
__device__ __forceinline__ void join_runs(const BeamParams &p, PickSpace &sp, int64_t row, int b) {
    const int lane = threadIdx.x & 31;
    const float2 *runs = p.runs + row * p.num_runs;
    const float cum = p.cum[row];
    const bool finished = p.finished && p.finished[row];
    // all at once up to 128 runs; those of a beam that is not live are of anything, and not used
    constexpr int kPer = 4;
    float2 r[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        r[k] = lane + 32 * k < p.num_runs ? runs[lane + 32 * k] : make_float2(-INFINITY, 0.f);
    float m = fmaxf(fmaxf(r[0].x, r[1].x), fmaxf(r[2].x, r[3].x));
    for (int i = lane + 32 * kPer; i < p.num_runs; i += 32) m = fmaxf(m, runs[i].x);
    m = warp_max(m);
    float s = 0.f, e = 0.f;
    // an empty run (its m -inf) has a sum of 0, or NaN
    auto add = [&](float2 run) {
        add_compensated(s, e, run.y * (run.x == m ? 1.f : exp2_approx((run.x - m) * kLog2e)));
    };
#pragma unroll
    for (int k = 0; k < kPer; ++k) add(r[k]);
    for (int i = lane + 32 * kPer; i < p.num_runs; i += 32) add(runs[i]);
    s += e;
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane) return;
    int kind = cum == -INFINITY ? kOut : finished ? kFinished : kLive;
    const bool bad = !(cum < INFINITY) || (kind == kLive && (!(m < INFINITY) || s != s));
    if (bad) atomicOr(p.status, kStatusInvalid);
    if (bad || (kind == kLive && m == -INFINITY)) kind = kOut;      // or every token is ruled out
    Offset offset = {0.f, cum, 0.f};
    if (kind == kLive) {
        // s = 2^n f with f within [0.7071, 1.4143), so that log f, off by its last place, is off by 2^-25 at most; n
        // log 2 in two parts, the first of 12 bits (its products with n are exact), and the sums with their errors
        int n;
        float f = frexpf(s, &n);
        if (f < 0.70710678f) f *= 2.f, n -= 1;
        constexpr float kLn2Hi = 0.693115234375f, kLn2Lo = static_cast<float>(0.69314718055994531 - 0.693115234375);
        const float large = -n * kLn2Hi, small = -n * kLn2Lo - logf(f);
        const float hi = cum + large, z = hi - cum;
        const float lo = (cum - (hi - z)) + (large - z) + small;
        const float top = hi + lo;
        offset = {m, top, lo - (top - hi)};
    }
    sp.kind[b] = kind;
    sp.offset[b] = offset;
    sp.shift[b] = kind == kLive ? make_float2(offset.top, offset.hi) : make_float2(0.f, -INFINITY);
    if (kind == kLive) atomicAdd(&sp.live, 1);
    if (kind != kOut) atomicMax(&sp.reach, __float_as_uint(fabsf(offset.hi)));
}

// One CTA a request.  The chunks that can be among the num_out first by their maxima, then the num_out first of
// those chunks' elements.  Most items are sorted out by a score in plain fp32, (x - top) + hi: two roundings,
// and lo left out, off by 2^-23 of |score| + |hi| at most.  Every thread belongs to one of a few groups, and the num_out-th largest of
// the groups' best scores is a bar that num_out items reach; an item below it by more than both may be off
// (2^-20 of |bar| + |hi|) cannot be among the first.  The few others get their key and are ranked by
// counting.  There are twice as many groups as num_out, at least a warp's lanes, so that the bar is seldom
// much below the num_out-th best item.  The chunks' bar holds for the elements too.
//
// Bound by latency: seven barriers, two loads in a row (the runs with the chunk maxima, the logits).  Shared
// memory is read side by side or by all alike, and the code is short: it runs once, from a cold cache.
template <typename T>
__device__ __forceinline__ void pick_request(const BeamParams &p, PickSpace &sp, int request) {
    constexpr int kPer = 4;                  // chunks that a thread keeps in registers
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int64_t row0 = static_cast<int64_t>(request) * p.num_beams;
    const int chunks = p.chunks, n = p.num_beams * chunks, most = p.num_out;
    const int groups = most <= 16 ? 32 : most <= 32 ? 64 : kGroups;
    const float *best = p.chunk_max + row0 * chunks;
    float x[kPer];
    auto fetch = [&](int base) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = base + k * kPickThreads + tid;
            x[k] = i < n ? best[i] : -INFINITY;
        }
    };
    fetch(0);
    if (tid < kGroups) sp.groups[tid] = 0;
    if (tid < 2) sp.count[tid] = 0;
    if (tid == 0) sp.bar = 0, sp.reach = 0, sp.live = 0;
    __syncthreads();
    for (int b = warp; b < p.num_beams; b += kPickThreads / 32) join_runs(p, sp, row0 + b, b);
    __syncthreads();
    auto beam_of = [&](int i) { return static_cast<int>(static_cast<uint64_t>(i) * p.per_chunk >> 40); };
    // the scores of the fetched chunks; -inf for nothing
    auto score = [&](int base) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const float2 shift = sp.shift[min(beam_of(base + k * kPickThreads + tid), p.num_beams - 1)];
            const float y = (x[k] - shift.x) + shift.y;
            x[k] = x[k] > -INFINITY && shift.y > -INFINITY ? y : -INFINITY;
        }
    };
    float first = -INFINITY;
    for (int base = 0; base < n; base += kPer * kPickThreads) {
        if (base) fetch(base);
        score(base);
#pragma unroll
        for (int k = 0; k < kPer; ++k) first = fmaxf(first, x[k]);
    }
    const bool ends = tid < p.num_beams && sp.kind[tid] == kFinished;      // this thread's finished beam
    if (ends) first = fmaxf(first, sp.offset[tid].hi);
    if (first > -INFINITY) atomicMax(&sp.groups[tid % groups], ordered(first));
    raise_bar(sp, groups, most);
    const float reach = __uint_as_float(sp.reach);
    auto below = [&](uint32_t bar) {         // what surely lies under a bar (0: there is none) lies under this
        const float y = float_of(bar);
        return bar ? y - (fabsf(y) + reach) * 0x1p-20f : -INFINITY;
    };
    float low = below(sp.bar);
    auto chunk = [&](int i) -> Ranked {
        const int b = beam_of(i);
        const uint32_t place = i;
        if (sp.kind[b] == kLive) return {key_of(best[i], sp.offset[b]), place};
        return {sp.kind[b] == kFinished && i == b * chunks ? key_of(0.f, sp.offset[b]) : 0, place};
    };
    for (int base = 0; base < n; base += kPer * kPickThreads) {
        if (n > kPer * kPickThreads) fetch(base), score(base);
        for (int k = 0; k < kPer; ++k) {
            const float y = k == 0 ? x[0] : k == 1 ? x[1] : k == 2 ? x[2] : x[3];
            if (!(y >= low) || y == -INFINITY) continue;
            const Ranked r = chunk(base + k * kPickThreads + tid);
            if (r.key) note(sp, 0, r.key, r.place);
        }
    }
    if (ends && sp.offset[tid].hi >= low) note(sp, 0, key_of(0.f, sp.offset[tid]), tid * chunks);
    __syncthreads();
    // the candidates themselves while they are few, else the first of them
    int kept = sp.count[0];
    const uint32_t *from = sp.place[0];
    if (kept > PA_MAX_BEAM_OUT) {
        kept = rank(sp, 0, n, most, chunk);
        from = sp.from;
        if (tid < kept) sp.from[tid] = sp.chosen[tid];
        if (kept == most) low = fmaxf(low, below(head_of(sp.chosen_key[most - 1])));
        __syncthreads();                             // sp.chosen is used again
    }
    // a pair's place in the order: beam, then token
    static_assert(PA_MAX_BEAM_VOCAB <= 1 << 24 && PA_MAX_BEAMS <= 1 << 8, "a beam and a token in 32 bits");
    const T *logits = static_cast<const T *>(p.logits) + row0 * p.row_stride;
    auto element = [&](int i) -> Ranked {
        const int c = static_cast<int>(from[i / kChunk]), b = beam_of(c);
        const uint32_t beam = static_cast<uint32_t>(b) << 24;
        if (sp.kind[b] == kFinished) return {i % kChunk ? 0 : key_of(0.f, sp.offset[b]), beam | p.end_token};
        const int token = (c - b * chunks) * kChunk + i % kChunk;
        if (token >= p.vocab) return {0, 0xffffffffu};
        return {key_of(static_cast<float>(logits[b * p.row_stride + token]), sp.offset[b]), beam | token};
    };
    // the scores of a lane's elements of chosen chunk k, and its beam's one item if that is finished
    auto scores_of = [&](int k, float (&y)[kChunk / 32]) {
        const int c = static_cast<int>(from[k]), b = beam_of(c);
        const float2 shift = sp.shift[b];
        const int token = (c - b * chunks) * kChunk + lane;
        const T *row = logits + b * p.row_stride + token;
#pragma unroll
        for (int i = 0; i < kChunk / 32; ++i)
            y[i] = token + 32 * i < p.vocab && shift.y > -INFINITY ? static_cast<float>(row[32 * i]) : -INFINITY;
#pragma unroll
        for (int i = 0; i < kChunk / 32; ++i)
            if (y[i] > -INFINITY) y[i] = (y[i] - shift.x) + shift.y;
        if (sp.kind[b] == kFinished && lane == 0) y[0] = sp.offset[b].hi;
    };
    float y[kChunk / 32];
    if (sp.live * chunks < 4 * most) {
        // of few chunks, the maximum of the num_out-th says little: the elements get a bar of their own
        if (tid < groups) sp.groups[tid] = 0;
        if (tid == 0) sp.bar = 0;
        __syncthreads();
        first = -INFINITY;
        for (int k = warp; k < kept; k += kPickThreads / 32) {
            scores_of(k, y);
#pragma unroll
            for (int i = 0; i < kChunk / 32; ++i) first = fmaxf(first, y[i]);
        }
        if (first > -INFINITY) atomicMax(&sp.groups[tid % groups], ordered(first));
        raise_bar(sp, groups, most);
        low = fmaxf(low, below(sp.bar));
    }
    for (int k = warp; k < kept; k += kPickThreads / 32) {
        scores_of(k, y);
        uint32_t passed = 0;
#pragma unroll
        for (int i = 0; i < kChunk / 32; ++i)
            if (y[i] > -INFINITY && y[i] >= low) passed |= 1u << i;
        for (; passed; passed &= passed - 1) {
            const Ranked r = element(k * kChunk + 32 * (__ffs(passed) - 1) + lane);
            if (r.key) note(sp, 1, r.key, r.place);
        }
    }
    __syncthreads();
    const int got = rank(sp, 1, kept * kChunk, most, element);
    if (tid < most) {
        const int64_t at = static_cast<int64_t>(request) * most + tid;
        const bool real = tid < got;
        const uint32_t place = sp.chosen[tid];
        p.scores[at] = real ? float_of(head_of(sp.chosen_key[tid])) : -INFINITY;
        p.beams[at] = real ? static_cast<int>(place >> 24) : -1;
        p.tokens[at] = real ? static_cast<int>(place & 0xffffffu) : -1;
    }
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const __grid_constant__ BeamParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ PickSpace sp;
    pick_request<T>(p, sp, blockIdx.x);
}

// Both in one launch: a cluster a request, whose first CTA picks when all have scanned.
template <typename T, bool VECTORS>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPickThreads)
    beam_small_kernel(const __grid_constant__ BeamParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ PickSpace sp;
    const int request = blockIdx.x / kCluster;
    const int w = blockIdx.x % kCluster * (kPickThreads / 32) + threadIdx.x / 32;
    const int beam = w / p.num_runs;
    if (beam < p.num_beams) scan_run<T, VECTORS>(p, request * p.num_beams + beam, w - beam * p.num_runs);
    __syncwarp();
    // the runs and chunk maxima of the cluster's other CTAs are there behind this barrier
    cluster_sync_all();
    if (blockIdx.x % kCluster == 0) pick_request<T>(p, sp, request);
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int64_t chunks_of(int vocab) { return (static_cast<int64_t>(vocab) + kChunk - 1) / kChunk; }

template <typename T>
cudaError_t launch_select(BeamParams &p, cudaStream_t stream) {
    const bool vectors = api_aligned(p.logits, 16) && p.row_stride % (16 / sizeof(T)) == 0;
    const int groups = (p.chunks + Eight<T>::kAhead - 1) / Eight<T>::kAhead;      // of a row, a warp's at least
    // A cluster's warps, with two groups each at most, for every request of one wave of clusters (16 fit; at 16
    // a call takes 9.4 us instead of 7).  One launch then saves 2.1 us of the host's 10.5, and costs the device 0.1 to
    // 1.6 us (4 beams x 32000 fp32 6.5 -> 7.1, 4 x 128000 bf16 7.4 -> 8.7, 16 x 128000 7.9 -> 9.5), which a stream that
    // waits for the host does not notice (one with work queued up does); a captured call has no host to wait for
    // and keeps its two launches.  The runs are the same, so the results are.
    const int warps = kCluster * kPickThreads / 32;
    if (p.num_requests <= kSmallRequests && p.num_beams * groups <= 2 * warps) {
        p.num_runs = groups < warps / p.num_beams ? groups : warps / p.num_beams;
        cudaStreamCaptureStatus status = cudaStreamCaptureStatusActive;
        if (cudaStreamIsCapturing(stream, &status) != cudaSuccess) (void)cudaGetLastError();
        if (status == cudaStreamCaptureStatusNone) {
            const dim3 grid(static_cast<unsigned>(p.num_requests * kCluster));
            return vectors ? launch_after(beam_small_kernel<T, true>, grid, kPickThreads, p, stream)
                           : launch_after(beam_small_kernel<T, false>, grid, kPickThreads, p, stream);
        }
    } else {
        // the rows in one wave of warps.  Rows are not divided unevenly: 2432 to 4863 of them leave up to half of the
        // warps idle, and past 4864 the last ones are read alone (32 beams x 16000 bf16: 76 requests 21.1 us, 77
        // 27.3, 152 32.7, 153 44.2)
        const int64_t per_row = kScanWarps / (static_cast<int64_t>(p.num_requests) * p.num_beams);
        p.num_runs = static_cast<int>(per_row < 1 ? 1 : per_row < groups ? per_row : groups);
    }
    const int64_t all = static_cast<int64_t>(p.num_requests) * p.num_beams * p.num_runs;
    const dim3 grid(static_cast<unsigned>((all + kScanThreads / 32 - 1) / (kScanThreads / 32)));
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
    if (static_cast<int64_t>(num_requests) * num_beams > INT32_MAX - kScanThreads)
        return api_fail(PA_ERR_UNSUPPORTED, "num_requests %d * num_beams %d", num_requests, num_beams);
    if (stride_row > (INT64_C(1) << 40))
        return api_fail(PA_ERR_UNSUPPORTED, "stride_row %lld", static_cast<long long>(stride_row));
    if (finished && (end_token < 0 || end_token >= vocab))
        return api_fail(PA_ERR_INVALID, "end_token %d not in [0, %d)", end_token, vocab);
    if (num_requests == 0) return PA_OK;
    if (!scores || !beams || !tokens || !logits || !cum_scores)
        return api_fail(PA_ERR_INVALID, "null pointer argument");
    const size_t elem = logits_dtype == PA_LOGITS_F32 ? 4 : 2;
    if (!api_aligned(logits, elem) || !api_aligned(scores, 4) || !api_aligned(beams, 4) || !api_aligned(tokens, 4) ||
        !api_aligned(cum_scores, 4))
        return api_fail(PA_ERR_INVALID, "logits, scores, beams, tokens or cum_scores are not aligned to their type");
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
    if (!workspace || !api_aligned(workspace, 256) ||
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
    // i < 2^21 chunks of a request and chunks <= 2^16: exact
    p.per_chunk = ((UINT64_C(1) << 40) + p.chunks - 1) / p.chunks;
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
