// pa_rope.cu -- rotary positions of q and k, alone and on the way into the paged cache.
//
// A pair of channels (x1, x2) of the token at position P turns by the angle P f_i of its pair i:
//   y1 = m (x1 cos - x2 sin), y2 = m (x2 cos + x1 sin),
// pairs (i, i + R/2) of the first R channels (half layout) or (2i, 2i + 1) (interleaved); the channels
// behind R pass through.
//
// Angles.  A position times a frequency in fp32 is off by 2^-24 of hundreds of thousands of radians.  The
// frequencies come as turns in 64-bit fixed point, F_i = f_i / 2 pi * 2^64: P F_i modulo 2^64 is the
// fraction of a turn, exact but for P times half a unit of F_i (2^-45 of a turn at a position of 2^20),
// and costs three integer products instead of fp64 ones.  Its top 32 bits, as an fp32 number of half turns
// (off by 2^-25 at most), go to sincospi.  Products and sums are fp32, each result is rounded once.
//
// Bound by memory: 2 bytes read and 2 written for each channel, a sincos per pair and token.  rope_kernel's
// CTAs go through the tokens with the next one's rows on their way (asynchronous copies into each thread's
// own shared memory) and its angles worked out, one pair a thread, while one token is turned.  A thread
// has two units of 16 channels in different heads at the same channels: they share a token's place and
// angles, and 64 bytes a thread are on their way.  16384 tokens of 32 + 8 heads of 128 channels: 54 us,
// 336 MB at 93 % of the copy rate; appended with 8 value heads 64 us (94 %), in E4M3 60 us (93 %); 7001
// tokens of 16 + 8 + 8 heads of 256 in E4M3, 64 channels interleaved: 33 us (90 %).  64 tokens: 1.9 us.
#include <cmath>
#include <cstring>
#include <numeric>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

enum { kRope = 0, kAppend = 1, kAppendFp8 = 2 };

constexpr int kMaxPairs = 128;
// rope_kernel: threads of a CTA, their units, tokens whose rows it has in hand or on their way.  Of 128 to
// 384 threads, 1 and 2 units and 2 to 4 stages the best.  CTAs of the most threads that an SM holds: 4 for bf16
// appends (16384 tokens 64.4 us against 66.4 with 3, 12000 46.3 against 48.7; as many at 28 + 4 and 64 + 8
// heads), 3 for rotations (54.0 against 55.3) and E4M3, which has no registers for 4 (33.4 against 36.3).
constexpr int kMaxThreads = 256;
constexpr int kUnits = 2;
constexpr int kStages = 2;
constexpr int ctas_per_sm(int kind) { return kind == kAppend ? 4 : 3; }
constexpr int kAnyChannels = 8192;           // of rope_any_kernel's CTA

struct Rows {                   // [token][head][head_dim] by element strides
    const void *base;
    int64_t token, head;
};

// A division by scale: factors a little under and over 1 / scale.
struct Quotient {
    float scale, low, high;
};

struct RopeParams {
    Rows q, k, v, q_out, k_out;          // v: append only; k_out: pa_rope only
    uint8_t *k_cache, *v_cache;
    const int64_t *positions, *slots;
    const uint64_t *turns;
    int64_t tokens, num_blocks, s_block, s_head, s_token;
    int nq, nk, nv, head_dim, pairs, inverse;
    float factor;
    Quotient k_by, v_by;
    int *status;
};

__device__ __forceinline__ float2 turn_of(uint64_t frequency, int64_t position, bool inverse, float factor) {
    const uint64_t turns = frequency * static_cast<uint64_t>(position);
    const float half_turns = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * factor, (inverse ? -s : s) * factor);
}

// Two fp32 in one register pair, for the instructions that work on both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}

__device__ __forceinline__ float2 split(uint64_t a) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
    return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ float2 floats_of(uint32_t two) {
    return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
}

__device__ __forceinline__ uint32_t bf16_of(float2 x) {
    uint32_t w;                          // the first source goes to the upper half
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(x.y), "f"(x.x));
    return w;
}

__device__ __forceinline__ uint32_t e4m3_of(float2 x) {
    uint16_t w;                          // the first source goes to the upper byte; saturated at +-448
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w) : "f"(x.y), "f"(x.x));
    return w;
}

// The E4M3 codes of x / scale, the quotient rounded to fp32 first, as the cache write makes them.  The
// factors lie 2^-21 to either side of 1 / scale, so the products enclose that quotient: where both have one
// code it is the quotient's, else (one pair in 2^15) the division decides.  A power of two has its
// reciprocal in both.
//   Here: the lower product's codes; bits in `unsure` where the other's differ.
__device__ __forceinline__ uint32_t codes_of(float2 x, const Quotient &by, uint32_t &unsure) {
    const uint64_t two = pair(x.x, x.y);
    const uint32_t w = e4m3_of(split(mul2(two, pair(by.low, by.low))));
    unsure |= w ^ e4m3_of(split(mul2(two, pair(by.high, by.high))));
    return w;
}

__device__ __forceinline__ uint8_t code_of_quotient(float x, float scale) {
    return static_cast<uint8_t>(e4m3_of(make_float2(__fdiv_rn(x, scale), 0.f)));
}

__device__ __forceinline__ const __nv_bfloat16 *row_of(const Rows &r, int64_t t, int h) {
    return static_cast<const __nv_bfloat16 *>(r.base) + t * r.token + h * r.head;
}

// Where head h of token t comes from: the query heads, the key heads, then the value heads.
template <int KIND>
__device__ __forceinline__ const __nv_bfloat16 *source(const RopeParams &p, int64_t t, int h) {
    if (h < p.nq) return row_of(p.q, t, h);
    h -= p.nq;
    if (KIND == kRope || h < p.nk) return row_of(p.k, t, h);
    return row_of(p.v, t, h - p.nk);
}

// Element offset of a slot in the pools, -1 for a token that is skipped (padding, or a slot outside the
// pool, which is flagged).
__device__ __forceinline__ int64_t place_of(const RopeParams &p, int64_t slot) {
    if (slot < 0) return -1;
    const int64_t page = slot >> 4;
    static_assert(kBlockSize == 16, "a slot's page");
    if (page >= p.num_blocks) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        return -1;
    }
    return page * p.s_block + static_cast<int>(slot & 15) * p.s_token;
}

// Copies the 16 bytes at `from` to shared memory when they arrive; several pend in committed groups.
__device__ __forceinline__ void send_for(uint4 *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}

// What a thread moves of every token: 16 channels of one head, in two vectors of eight.
struct Unit {
    const __nv_bfloat16 *from;               // at token 0
    uint8_t *to;                             // a row at token 0, or the head's rows in the pool
    int from_token, to_token;                // strides in elements
    bool live, to_rows, is_k, turned;
};

// Half layout with pairs a multiple of 8, and every interleaved one.  Grid: x = tokens (each CTA takes every
// gridDim.x-th), y = groups of heads, kUnits * blockDim.x units each.  A thread's units lie in different
// heads but at the same channels, so that they share the token's place and angles.
// PARTIAL: a vector may hold interleaved pairs of which some turn and some do not.
template <int KIND, bool INTERLEAVED, bool PARTIAL>
__global__ void __launch_bounds__(kMaxThreads, ctas_per_sm(KIND)) rope_kernel(const __grid_constant__ RopeParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ uint4 rows[];                  // [kStages][kUnits][2][threads]
    // two pairs' (cos, cos, sin, sin), where the reads of a warp's units fall side by side
    __shared__ float4 turns[2][kMaxPairs / 2];
    auto turns_at = [](int i) {              // of pairs i (even) and i + 1
        return INTERLEAVED ? i / 2 % 2 * (kMaxPairs / 4) + i / 4 : i % 8 / 2 * (kMaxPairs / 8) + i / 8;
    };
    constexpr int kElem = KIND == kAppendFp8 ? 1 : 2;
    const int tid = threadIdx.x, threads = blockDim.x;
    auto mine_at = [&](int stage, int k) { return rows + ((stage * kUnits + k) * 2) * threads + tid; };
    const int per_head = p.head_dim / 16;            // 4, 8 or 16: blockDim.x is a multiple of it
    const int u = tid & (per_head - 1);
    // the unit's two vectors of 8 channels: those of 8 pairs; interleaved, one in either half of the head;
    // of the channels behind the turned ones, one in either half of them.  Neighbouring threads' are adjacent.
    const bool paired = !INTERLEAVED && 8 * u < p.pairs;
    const int c0 = INTERLEAVED || paired ? 8 * u : p.pairs + 8 * u;
    const int c1 = (paired ? p.pairs : p.head_dim / 2) + 8 * u;
    Unit unit[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        Unit &x = unit[k];
        int head = ((blockIdx.y * kUnits + k) * threads + tid) / per_head;
        x.live = head < p.nq + p.nk + p.nv;
        const bool is_q = head < p.nq;
        x.is_k = !is_q && (KIND == kRope || head < p.nq + p.nk);
        x.to_rows = KIND == kRope || is_q;
        x.turned = (is_q || x.is_k) && (INTERLEAVED ? 4 * u < p.pairs : paired);
        head -= is_q ? 0 : x.is_k ? p.nq : p.nq + p.nk;
        const Rows &from = is_q ? p.q : x.is_k ? p.k : p.v, &to = is_q ? p.q_out : p.k_out;
        x.from = static_cast<const __nv_bfloat16 *>(from.base) + head * from.head + c0;
        x.from_token = static_cast<int>(from.token);
        x.to_token = static_cast<int>(to.token);
        x.to = x.to_rows ? static_cast<uint8_t *>(const_cast<void *>(to.base)) + (head * to.head + c0) * 2
                         : (x.is_k ? p.k_cache : p.v_cache) + (head * p.s_head + c0) * kElem;
    }
    const int apart = c1 - c0;

    // which pair's angle this thread works out; it moves from token to token, so that all warps take part
    int mine = tid;
    auto work_out = [&](int buffer, int64_t position) {
        for (int i = mine; i < p.pairs; i += threads) {
            const float2 w = turn_of(p.turns[i], position, p.inverse != 0, p.factor);
            float *four = reinterpret_cast<float *>(&turns[buffer][turns_at(i & ~1)]);
            four[i % 2] = w.x;
            four[2 + i % 2] = w.y;
        }
        mine += p.pairs;
        while (mine >= threads) mine -= threads;
    };
    const int tokens = static_cast<int>(p.tokens), step = gridDim.x;
    int sent = blockIdx.x;                           // tokens <= 2^30, and so is step
    auto send = [&](int stage) {
        if (sent < tokens) {
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                if (!unit[k].live) continue;
                const __nv_bfloat16 *from = unit[k].from + static_cast<int64_t>(sent) * unit[k].from_token;
                send_for(mine_at(stage, k), from);
                send_for(mine_at(stage, k) + threads, from + apart);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        sent += step;
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) send(s);
    int t = blockIdx.x;
    int64_t slot = KIND == kRope ? 0 : p.slots[t];
    work_out(0, p.positions[t]);
    int64_t position = t + step < tokens ? p.positions[t + step] : 0;
    __syncthreads();
    for (int buffer = 0, stage = 0; t < tokens; buffer ^= 1, t += step) {
        send(stage == 0 ? kStages - 1 : stage - 1);
        const int64_t now = slot;
        if (t + step < tokens) {
            if (KIND != kRope) slot = p.slots[t + step];
            work_out(buffer ^ 1, position);
            if (t + 2 * step < tokens) position = p.positions[t + 2 * step];
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        const int64_t at = KIND == kRope ? 0 : place_of(p, now);
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            if (!unit[k].live || at < 0) continue;
            const uint4 a4 = *mine_at(stage, k), b4 = mine_at(stage, k)[threads];
            uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
            const bool codes = KIND == kAppendFp8 && !unit[k].to_rows, turned = unit[k].turned;
            float2 x[4], y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = floats_of(a[j]), y[j] = floats_of(b[j]);
            if (!INTERLEAVED && turned) {
                // two pairs: one half of each in a word of a, the other in that of b
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 cs = turns[buffer][turns_at(8 * u + 2 * j)];
                    const uint64_t x2 = pair(x[j].x, x[j].y), y2 = pair(y[j].x, y[j].y), c2 = pair(cs.x, cs.y);
                    const uint64_t s2 = pair(cs.z, cs.w), n2 = pair(-cs.z, -cs.w);
                    x[j] = split(fma2(x2, c2, mul2(y2, n2)));
                    y[j] = split(fma2(y2, c2, mul2(x2, s2)));
                }
            }
            if (INTERLEAVED && turned) {
                // a pair a word
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int first = c0 / 2 + v * (apart / 2), pairs = p.pairs - first;
                    if (pairs <= 0) continue;
                    const float4 cs[2] = {turns[buffer][turns_at(first)], turns[buffer][turns_at(first + 2)]};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (PARTIAL && j >= pairs) continue;
                        float2 &z = v ? y[j] : x[j];
                        const float c = j % 2 ? cs[j / 2].y : cs[j / 2].x, s = j % 2 ? cs[j / 2].w : cs[j / 2].z;
                        z = make_float2(__fmaf_rn(z.x, c, -z.y * s), __fmaf_rn(z.y, c, z.x * s));
                    }
                }
            }
            uint32_t unsure = 0;
            if (codes) {
                const Quotient &by = unit[k].is_k ? p.k_by : p.v_by;
#pragma unroll
                for (int j = 0; j < 4; ++j) a[j] = codes_of(x[j], by, unsure), b[j] = codes_of(y[j], by, unsure);
            } else if (turned) {
#pragma unroll
                for (int j = 0; j < 4; ++j) a[j] = bf16_of(x[j]), b[j] = bf16_of(y[j]);
            }
            uint8_t *to = unit[k].to + (unit[k].to_rows ? static_cast<int64_t>(t) * unit[k].to_token * 2 : at * kElem);
            if (codes && unsure) {
                // seldom: one channel after another, its value once more and divided
                const float scale = unit[k].is_k ? p.k_by.scale : p.v_by.scale;
                const __nv_bfloat16 *near = reinterpret_cast<const __nv_bfloat16 *>(mine_at(stage, k));
                const __nv_bfloat16 *far = near + 8 * threads;
#pragma unroll 1
                for (int e = 0; e < 16; ++e) {
                    const bool back = INTERLEAVED ? e & 1 : e >= 8;        // the pair's second channel
                    const int of_pair = INTERLEAVED ? (e < 8 ? c0 / 2 : c1 / 2 - 4) + e / 2 : 8 * u + e % 8;
                    float x = __bfloat162float(e < 8 ? near[e] : far[e - 8]);
                    if (unit[k].turned && of_pair < p.pairs) {
                        const int o = INTERLEAVED ? e ^ 1 : e ^ 8;
                        const float y = __bfloat162float(o < 8 ? near[o] : far[o - 8]);
                        const float *cs = reinterpret_cast<const float *>(&turns[buffer][turns_at(of_pair & ~1)]) + of_pair % 2;
                        x = __fmaf_rn(x, cs[0], __fmul_rn(y, back ? cs[2] : -cs[2]));
                    }
                    to[e < 8 ? e : apart + e - 8] = code_of_quotient(x, scale);
                }
            } else if (codes) {
                *reinterpret_cast<uint2 *>(to) = make_uint2(a[0] | a[1] << 16, a[2] | a[3] << 16);
                *reinterpret_cast<uint2 *>(to + apart) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
            } else {
                *reinterpret_cast<uint4 *>(to) = make_uint4(a[0], a[1], a[2], a[3]);
                *reinterpret_cast<uint4 *>(to + apart * 2) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        }
        __syncthreads();                             // the next angles are there, these no longer read
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
}

// Half layout with any other number of pairs, where the second channel of a pair starts at any 2 bytes.
// Grid: x = tokens, y = groups of heads.  The heads' rows lie in shared memory whole; a thread makes eight
// neighbouring results, each from its own channel and the one it is paired with.  Bound by issue (82 %
// busy, 280 instructions a warp's 32 vectors): 93 us for 100 of 128 channels of the 16384 tokens above.
template <int KIND>
__global__ void __launch_bounds__(256) rope_any_kernel(const __grid_constant__ RopeParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ uint4 rows[kAnyChannels / 8];
    // of pair i at [i % 8][i / 8]: neighbouring threads read side by side
    __shared__ float2 turns[8][kMaxPairs / 8 + 1];
    const int64_t t = blockIdx.x;
    const int64_t at = KIND == kRope ? 0 : place_of(p, p.slots[t]);
    if (at < 0) return;                              // the whole CTA
    const int head_bits = p.head_dim == 64 ? 3 : p.head_dim == 128 ? 4 : 5;      // a head's vectors
    const int per_cta = (kAnyChannels / 8) >> head_bits, first = blockIdx.y * per_cta;
    const int vectors = min(per_cta, p.nq + p.nk + p.nv - first) << head_bits;
    for (int i = threadIdx.x; i < vectors; i += blockDim.x)
        send_for(rows + i, source<KIND>(p, t, first + (i >> head_bits)) + (i & ((1 << head_bits) - 1)) * 8);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int64_t position = p.positions[t];
    for (int i = threadIdx.x; i < p.pairs; i += blockDim.x)
        turns[i % 8][i / 8] = turn_of(p.turns[i], position, p.inverse != 0, p.factor);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    // a thread's channels are the same in all its heads: blockDim.x is a multiple of a head's vectors
    const int c0 = (threadIdx.x & ((1 << head_bits) - 1)) * 8;
    // for each channel its partner (itself: not turned), and its own and the partner's factor
    int partner[8];
    float2 cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = c0 + j, i = c < p.pairs ? c : c - p.pairs;
        const bool turned = c < 2 * p.pairs;
        partner[j] = turned ? (c < p.pairs ? c + p.pairs : i) : c;
        cs[j] = turned ? turns[i & 7][i >> 3] : make_float2(1.f, 0.f);
        if (c < p.pairs) cs[j].y = -cs[j].y;
    }
    for (int i = threadIdx.x; i < vectors; i += blockDim.x) {
        const int h = first + (i >> head_bits);
        const uint4 own = rows[i];
        const uint32_t w[4] = {own.x, own.y, own.z, own.w};
        const __nv_bfloat16 *row = reinterpret_cast<const __nv_bfloat16 *>(rows) + (i >> head_bits) * p.head_dim;
        float2 y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = floats_of(w[j]);
        if (h < p.nq + p.nk) {                       // values are not turned
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float &x = j % 2 ? y[j / 2].y : y[j / 2].x;
                const float turn = __fmaf_rn(x, cs[j].x, __bfloat162float(row[partner[j]]) * cs[j].y);
                if (partner[j] != c0 + j) x = turn;
            }
        }
        if (KIND == kRope || h < p.nq) {
            const __nv_bfloat16 *to = h < p.nq ? row_of(p.q_out, t, h) : row_of(p.k_out, t, h - p.nq);
            *reinterpret_cast<uint4 *>(const_cast<__nv_bfloat16 *>(to) + c0) =
                make_uint4(bf16_of(y[0]), bf16_of(y[1]), bf16_of(y[2]), bf16_of(y[3]));
            continue;
        }
        const bool is_k = h < p.nq + p.nk;
        uint8_t *pool = is_k ? p.k_cache : p.v_cache;
        const int64_t to = at + (h - p.nq - (is_k ? 0 : p.nk)) * p.s_head + c0;
        if (KIND == kAppendFp8) {
            const Quotient &by = is_k ? p.k_by : p.v_by;
            uint32_t c[4], unsure = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = codes_of(y[j], by, unsure);
            *reinterpret_cast<uint2 *>(pool + to) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
            if (unsure)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    pool[to + j] = code_of_quotient(j % 2 ? y[j / 2].y : y[j / 2].x, by.scale);
        } else if (is_k) {
            *reinterpret_cast<uint4 *>(pool + to * 2) =
                make_uint4(bf16_of(y[0]), bf16_of(y[1]), bf16_of(y[2]), bf16_of(y[3]));
        } else {
            *reinterpret_cast<uint4 *>(pool + to * 2) = own;
        }
    }
}

template <int KIND>
cudaError_t launch_rope(const RopeParams &p, bool interleaved, cudaStream_t stream) {
    const int channels = (p.nq + p.nk + p.nv) * p.head_dim;
    if (!interleaved && p.pairs % 8)
        return launch_after(rope_any_kernel<KIND>,
                            dim3(static_cast<unsigned>(p.tokens),
                                 static_cast<unsigned>((channels + kAnyChannels - 1) / kAnyChannels)),
                            256, p, stream);
    const int units = (channels / 16 + kUnits - 1) / kUnits;
    const int groups = (units + kMaxThreads - 1) / kMaxThreads;
    const int threads = ((units + groups - 1) / groups + 31) / 32 * 32;
    // one wave: ctas_per_sm of the largest CTAs, or as many threads in smaller ones, fit an SM
    const int fit = ctas_per_sm(KIND) * kMaxThreads / threads, per_sm = fit < 32 ? fit : 32;
    const int64_t wave = (152 * per_sm + groups - 1) / groups;
    const dim3 grid(static_cast<unsigned>(p.tokens < wave ? p.tokens : wave), static_cast<unsigned>(groups));
    const size_t rows = static_cast<size_t>(kStages) * kUnits * 2 * threads * sizeof(uint4);
    if (!interleaved) return launch_after(rope_kernel<KIND, false, false>, grid, threads, p, stream, rows);
    return p.pairs % 4 ? launch_after(rope_kernel<KIND, true, true>, grid, threads, p, stream, rows)
                       : launch_after(rope_kernel<KIND, true, false>, grid, threads, p, stream, rows);
}

// ---- argument checks --------------------------------------------------------------------

// The elements of a [tokens][heads][head_dim] tensor in two levels: `outer` steps of runs that span
// `span` elements.  Every row (of head_dim) starts a whole number of `period`s behind the first; 0 where there is
// one row.  The stride of an axis of length 1 counts as none.
struct Extent {
    uintptr_t at;
    int64_t outer, count, span, period, row;     // bytes but for count
};

Extent extent_of(const Rows &r, int64_t tokens, int heads, int head_dim) {
    const int64_t st = tokens > 1 ? r.token : 0, sh = heads > 1 ? r.head : 0;
    const bool by_token = st >= sh;
    Extent e;
    e.at = reinterpret_cast<uintptr_t>(r.base);
    e.outer = 2 * (by_token ? st : sh);
    e.count = by_token ? tokens : heads;
    e.span = 2 * ((by_token ? (heads - 1) * sh : (tokens - 1) * st) + head_dim);
    e.period = 2 * std::gcd(st, sh);
    e.row = 2 * head_dim;
    return e;
}

// False where the two are seen to share no element: apart as a whole; with the same outer stride and
// runs beside one another (the slices of one projection's rows); or with rows beside one another in a period
// that both keep (the slices of each head's part of a projection).
bool may_overlap(const Extent &a, const Extent &b) {
    const uintptr_t a_end = a.at + (a.count - 1) * a.outer + a.span, b_end = b.at + (b.count - 1) * b.outer + b.span;
    if (a_end <= b.at || b_end <= a.at) return false;
    // whether runs of a and b, every s bytes, lie beside one another
    auto beside = [&](int64_t s, int64_t run_a, int64_t run_b) {
        if (s == 0) return false;
        const uintptr_t u = static_cast<uintptr_t>(s);
        const int64_t d = static_cast<int64_t>(b.at >= a.at ? (b.at - a.at) % u : (u - (a.at - b.at) % u) % u);
        return d >= run_a && d + run_b <= s;
    };
    if (a.outer == b.outer && beside(a.outer, a.span, b.span)) return false;
    return !beside(std::gcd(a.period, b.period), a.row, b.row);
}

int check_rows(const char *name, const Rows &r, int64_t tokens, int heads, int head_dim, bool written) {
    if (!r.base || !api_aligned(r.base, 16))
        return api_fail(PA_ERR_INVALID, "%s is NULL or not 16-byte aligned", name);
    const int64_t st = tokens > 1 ? r.token : 0, sh = heads > 1 ? r.head : 0;
    constexpr int64_t kMost = INT64_C(1) << 40;      // far beyond memory: offsets stay within 64 bits
    if (st < 0 || sh < 0 || st % 8 || sh % 8 || st > kMost || sh > kMost)
        return api_fail(PA_ERR_INVALID, "%s: strides (%lld, %lld) must be multiples of 16 bytes, not negative", name,
                        static_cast<long long>(r.token), static_cast<long long>(r.head));
    if (st > INT32_MAX)
        return api_fail(PA_ERR_UNSUPPORTED, "%s: token stride %lld", name, static_cast<long long>(st));
    if (!written) return PA_OK;
    const Extent e = extent_of(r, tokens, heads, head_dim);
    const int64_t inner = st >= sh ? sh : st, inner_count = st >= sh ? heads : tokens;
    if ((inner_count > 1 && inner < head_dim) || (e.count > 1 && e.outer < e.span))
        return api_fail(PA_ERR_INVALID, "%s: rows overlap (strides %lld, %lld)", name, static_cast<long long>(r.token),
                        static_cast<long long>(r.head));
    return PA_OK;
}

bool same_rows(const Rows &a, const Rows &b, int64_t tokens, int heads) {
    return a.base == b.base && (tokens <= 1 || a.token == b.token) && (heads <= 1 || a.head == b.head);
}

int check_common(int64_t num_tokens, int nq, int nk, int head_dim, int rotary_dim, float factor) {
    if (num_tokens < 0) return api_fail(PA_ERR_INVALID, "num_tokens %lld", static_cast<long long>(num_tokens));
    if (num_tokens > (INT64_C(1) << 30))
        return api_fail(PA_ERR_UNSUPPORTED, "num_tokens %lld > 2^30", static_cast<long long>(num_tokens));
    if (nq < 0 || nk < 0) return api_fail(PA_ERR_INVALID, "head counts (%d, %d)", nq, nk);
    if (nq > 65536 || nk > 65536) return api_fail(PA_ERR_UNSUPPORTED, "head counts (%d, %d) > 65536", nq, nk);
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return api_fail(PA_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", head_dim);
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim)
        return api_fail(PA_ERR_INVALID, "rotary_dim %d must be even, from 2 to head_dim %d", rotary_dim, head_dim);
    if (!std::isfinite(factor)) return api_fail(PA_ERR_INVALID, "attention_factor %g", static_cast<double>(factor));
    return PA_OK;
}

// Outside the range where the factors and products are sure to be normal numbers, factors that never
// agree: every quotient is divided.
Quotient quotient_by(float scale) {
    int n;
    const bool exact = std::frexp(scale, &n) == 0.5f;
    if (!(n > -100 && n < 100)) return {scale, -1.f, 1.f};
    const double inverse = 1.0 / scale;
    return {scale, static_cast<float>(exact ? inverse : inverse * (1 - 0x1p-21)),
            static_cast<float>(exact ? inverse : inverse * (1 + 0x1p-21))};
}

// Number of a pair that makes `turns` full turns within `len` positions, as a real number.
double pair_of_turns(double turns, int rotary_dim, double base, double len) {
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    return rotary_dim * std::log(len / (turns * kTwoPi)) / (2 * std::log(base));
}

// ---- frequencies, in twice a double's bits: an entry holds up to 62 of a frequency ---------

// hi + lo, lo at most half a unit in hi's last place.
struct Wide {
    double hi, lo;
};

Wide plus(const Wide &a, const Wide &b) {
    const double s = a.hi + b.hi, z = s - a.hi;
    const double rest = (a.hi - (s - z)) + (b.hi - z) + (a.lo + b.lo);
    const double hi = s + rest;
    return {hi, rest - (hi - s)};
}

Wide times(const Wide &a, const Wide &b) {
    const double x = a.hi * b.hi;
    const double rest = std::fma(a.hi, b.hi, -x) + (a.hi * b.lo + a.lo * b.hi);
    const double hi = x + rest;
    return {hi, rest - (hi - x)};
}

Wide over(const Wide &a, const Wide &b) {
    const double q = a.hi / b.hi;
    const Wide left = plus(a, times(b, {-q, 0.0}));
    return plus({q, 0.0}, {left.hi / b.hi, 0.0});
}

// The n-th root of b > 0: one step of Newton's iteration from the root in a double.  Where its powers or their
// rounding errors leave a double's range the double stands.
Wide root(double b, int n) {
    const double x = std::pow(b, 1.0 / n);
    if (std::fabs(std::log2(b)) > 900) return {x, 0.0};
    Wide power = {x, 0.0};
    for (int i = 1; i < n; ++i) power = times(power, {x, 0.0});
    const Wide off = plus(over(power, {b, 0.0}), {-1.0, 0.0});        // n times the relative error
    return plus({x, 0.0}, {-x * off.hi / n, 0.0});
}

// 1 / 2 pi, to 2^-165.
constexpr double kTurnsPerRadian[3] = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57, -0x1.6447e493ad4cep-111};

// x modulo 1 in units of 2^-128.
unsigned __int128 fraction_of(double x) {
    int e;
    const double m = std::frexp(std::fabs(x), &e);
    unsigned __int128 u = static_cast<uint64_t>(std::ldexp(m, 53));
    e += 128 - 53;
    u = e >= 128 ? 0 : e >= 0 ? u << e : e > -128 ? u >> -e : 0;
    return x < 0 ? 0 - u : u;
}

unsigned __int128 fraction_of_product(double a, double b) {
    const double x = a * b;
    return fraction_of(x) + fraction_of(std::fma(a, b, -x));
}

// The table's entries: f radians a position as turns, the nearest multiple of 2^-64.
int write_turns(uint64_t *turns_h, const Wide *f, int num_pairs) {
    if (!turns_h) return api_fail(PA_ERR_INVALID, "null pointer argument");
    for (int i = 0; i < num_pairs; ++i)
        if (!std::isfinite(f[i].hi) || !std::isfinite(f[i].lo))
            return api_fail(PA_ERR_INVALID, "frequency %d is not finite", i);
    for (int i = 0; i < num_pairs; ++i) {
        unsigned __int128 u = 0;
        for (double part : {f[i].hi, f[i].lo})
            for (double by : kTurnsPerRadian) u += fraction_of_product(part, by);
        turns_h[i] = static_cast<uint64_t>((u + (static_cast<unsigned __int128>(1) << 63)) >> 64);
    }
    return PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" int pa_rope_table_of(uint64_t *turns_h, const double *frequencies_h, int num_pairs) {
    using namespace pa;
    if (num_pairs < 1 || num_pairs > kMaxPairs)
        return api_fail(PA_ERR_INVALID, "num_pairs %d not in [1, %d]", num_pairs, kMaxPairs);
    if (!turns_h || !frequencies_h) return api_fail(PA_ERR_INVALID, "null pointer argument");
    Wide f[kMaxPairs];
    for (int i = 0; i < num_pairs; ++i) f[i] = {frequencies_h[i], 0.0};
    return write_turns(turns_h, f, num_pairs);
}

extern "C" int pa_rope_table(uint64_t *turns_h, float *attention_factor_h, int rotary_dim, double base, int scaling,
                             double factor, double low, double high, int64_t original_len) {
    using namespace pa;
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 2 * kMaxPairs)
        return api_fail(PA_ERR_INVALID, "rotary_dim %d must be even, from 2 to %d", rotary_dim, 2 * kMaxPairs);
    if (!(base > 1) || !std::isfinite(base)) return api_fail(PA_ERR_INVALID, "base %g must be above 1", base);
    if (scaling < PA_ROPE_NONE || scaling > PA_ROPE_YARN) return api_fail(PA_ERR_UNSUPPORTED, "scaling %d", scaling);
    if (scaling != PA_ROPE_NONE && (!(factor > 0) || !std::isfinite(factor)))
        return api_fail(PA_ERR_INVALID, "scaling factor %g must be positive and finite", factor);
    if (scaling == PA_ROPE_NTK && rotary_dim == 2)
        return api_fail(PA_ERR_INVALID, "rotary_dim 2 has no second frequency for a scaled base");
    if (scaling == PA_ROPE_BANDS || scaling == PA_ROPE_YARN) {
        if (!(low > 0) || !(high > low) || !std::isfinite(high))
            return api_fail(PA_ERR_INVALID, "low %g, high %g must be positive and ascend", low, high);
        if (original_len <= 0)
            return api_fail(PA_ERR_INVALID, "original_len %lld", static_cast<long long>(original_len));
    }
    const int n = rotary_dim / 2;
    const double len = static_cast<double>(original_len);
    // base^(-i / n) as the powers of the n-th root; the scaled base's as those of two roots,
    // (base s^(n / (n - 1)))^(-i / n) = base^(-i / n) s^(-i / (n - 1))
    Wide step = over({1.0, 0.0}, root(base, n)), f[kMaxPairs];
    if (scaling == PA_ROPE_NTK) step = times(step, over({1.0, 0.0}, root(factor, n - 1)));
    f[0] = {1.0, 0.0};
    for (int i = 1; i < n; ++i) f[i] = times(f[i - 1], step);
    // f / factor where r is 0, f where it is 1
    auto between = [&](const Wide &x, Wide r) {
        r = r.hi <= 0 ? Wide{0.0, 0.0} : r.hi >= 1 ? Wide{1.0, 0.0} : r;
        return times(x, plus(over(plus({1.0, 0.0}, {-r.hi, -r.lo}), {factor, 0.0}), r));
    };
    float m = 1.f;
    if (scaling == PA_ROPE_LINEAR) {
        for (int i = 0; i < n; ++i) f[i] = over(f[i], {factor, 0.0});
    } else if (scaling == PA_ROPE_BANDS) {
        for (int i = 0; i < n; ++i) {
            const Wide turns = times(times(f[i], {len, 0.0}), {kTurnsPerRadian[0], kTurnsPerRadian[1]});
            f[i] = between(f[i], over(plus(turns, {-low, 0.0}), plus({high, 0.0}, {-low, 0.0})));
        }
    } else if (scaling == PA_ROPE_YARN) {
        const double first = std::fmax(std::floor(pair_of_turns(high, rotary_dim, base, len)), 0.0);
        const double last = std::fmin(std::ceil(pair_of_turns(low, rotary_dim, base, len)), rotary_dim - 1.0);
        for (int i = 0; i < n; ++i)
            f[i] = between(f[i], plus({1.0, 0.0}, over({first - i, 0.0}, {std::fmax(last - first, 0.001), 0.0})));
        if (factor > 1) m = static_cast<float>(0.1 * std::log(factor) + 1);
    }
    const int rc = write_turns(turns_h, f, n);
    if (rc == PA_OK && attention_factor_h) *attention_factor_h = m;
    return rc;
}

extern "C" int pa_rope(void *q_out, void *k_out, const void *q, const void *k, const int64_t *positions,
                       const uint64_t *turns, int64_t num_tokens, int num_q_heads, int num_k_heads, int head_dim,
                       int rotary_dim, int64_t q_out_stride_token, int64_t q_out_stride_head,
                       int64_t k_out_stride_token, int64_t k_out_stride_head, int64_t q_stride_token,
                       int64_t q_stride_head, int64_t k_stride_token, int64_t k_stride_head, int interleaved,
                       int inverse, float attention_factor, void *stream) {
    using namespace pa;
    int rc = check_common(num_tokens, num_q_heads, num_k_heads, head_dim, rotary_dim, attention_factor);
    if (rc) return rc;
    if (num_tokens == 0 || num_q_heads + num_k_heads == 0) return PA_OK;
    if (!positions || !turns) return api_fail(PA_ERR_INVALID, "null pointer argument");
    if (!api_aligned(positions, 8) || !api_aligned(turns, 8))
        return api_fail(PA_ERR_INVALID, "positions and turns must be 8-byte aligned");
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    p.q = {q, q_stride_token, q_stride_head};
    p.k = {k, k_stride_token, k_stride_head};
    p.q_out = {q_out, q_out_stride_token, q_out_stride_head};
    p.k_out = {k_out, k_out_stride_token, k_out_stride_head};
    const struct {
        const char *name;
        const Rows *of, *to;
        int heads;
    } both[2] = {{"q", &p.q, &p.q_out, num_q_heads}, {"k", &p.k, &p.k_out, num_k_heads}};
    for (const auto &x : both) {
        if (x.heads == 0) continue;
        rc = check_rows(x.name, *x.of, num_tokens, x.heads, head_dim, false);
        if (rc) return rc;
        rc = check_rows(x.of == &p.q ? "q_out" : "k_out", *x.to, num_tokens, x.heads, head_dim, true);
        if (rc) return rc;
    }
    for (const auto &x : both)          // an output over an input: only its own, in place
        for (const auto &y : both) {
            if (x.heads == 0 || y.heads == 0) continue;
            const Extent to = extent_of(*x.to, num_tokens, x.heads, head_dim);
            if (!(x.of == y.of && same_rows(*x.to, *x.of, num_tokens, x.heads)) &&
                may_overlap(to, extent_of(*y.of, num_tokens, y.heads, head_dim)))
                return api_fail(PA_ERR_INVALID, "%s_out overlaps %s (only in place, with the same strides)", x.name, y.name);
            if (x.of != y.of && may_overlap(to, extent_of(*y.to, num_tokens, y.heads, head_dim)))
                return api_fail(PA_ERR_INVALID, "q_out and k_out overlap");
        }
    p.tokens = num_tokens;
    p.positions = positions;
    p.turns = turns;
    p.nq = num_q_heads;
    p.nk = num_k_heads;
    p.head_dim = head_dim;
    p.pairs = rotary_dim / 2;
    p.inverse = inverse ? 1 : 0;
    p.factor = attention_factor;
    const cudaError_t e = launch_rope<kRope>(p, interleaved != 0, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : api_cuda_fail(e, "rope launch");
}

extern "C" int pa_rope_append(void *q_out, const void *q, const void *k, const void *v, void *k_cache, void *v_cache,
                              const int64_t *slot_mapping, const int64_t *positions, const uint64_t *turns,
                              int64_t num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
                              int block_size, int64_t num_blocks, int64_t q_out_stride_token,
                              int64_t q_out_stride_head, int64_t q_stride_token, int64_t q_stride_head,
                              int64_t k_stride_token, int64_t k_stride_head, int64_t v_stride_token,
                              int64_t v_stride_head, int64_t stride_block, int64_t stride_head,
                              int64_t stride_token, int interleaved, float attention_factor, int kv_dtype,
                              float k_scale, float v_scale, void *stream) {
    using namespace pa;
    int rc = check_common(num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim, attention_factor);
    if (rc) return rc;
    if (num_kv_heads == 0) return api_fail(PA_ERR_INVALID, "num_kv_heads 0");
    rc = api_check_kv_dtype(kv_dtype, k_scale, v_scale);
    if (rc) return rc;
    rc = api_check_pool(head_dim, block_size, num_blocks, num_kv_heads, stride_block, stride_head, stride_token,
                        kv_dtype);
    if (rc) return rc;
    if (num_tokens == 0) return PA_OK;
    if (!positions || !turns || !slot_mapping || !k_cache || !v_cache)
        return api_fail(PA_ERR_INVALID, "null pointer argument");
    if (!api_aligned(positions, 8) || !api_aligned(turns, 8) || !api_aligned(slot_mapping, 8))
        return api_fail(PA_ERR_INVALID, "positions, slot_mapping and turns must be 8-byte aligned");
    if (!api_aligned(k_cache, 16) || !api_aligned(v_cache, 16))
        return api_fail(PA_ERR_INVALID, "the KV pools must be 16-byte aligned");
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    p.q = {q, q_stride_token, q_stride_head};
    p.k = {k, k_stride_token, k_stride_head};
    p.v = {v, v_stride_token, v_stride_head};
    p.q_out = {q_out, q_out_stride_token, q_out_stride_head};
    rc = check_rows("k", p.k, num_tokens, num_kv_heads, head_dim, false);
    if (rc) return rc;
    rc = check_rows("v", p.v, num_tokens, num_kv_heads, head_dim, false);
    if (rc) return rc;
    if (num_q_heads > 0) {
        rc = check_rows("q", p.q, num_tokens, num_q_heads, head_dim, false);
        if (rc) return rc;
        rc = check_rows("q_out", p.q_out, num_tokens, num_q_heads, head_dim, true);
        if (rc) return rc;
        const Extent to = extent_of(p.q_out, num_tokens, num_q_heads, head_dim);
        if (!same_rows(p.q_out, p.q, num_tokens, num_q_heads) &&
            may_overlap(to, extent_of(p.q, num_tokens, num_q_heads, head_dim)))
            return api_fail(PA_ERR_INVALID, "q_out overlaps q (only in place, with the same strides)");
        if (may_overlap(to, extent_of(p.k, num_tokens, num_kv_heads, head_dim)) ||
            may_overlap(to, extent_of(p.v, num_tokens, num_kv_heads, head_dim)))
            return api_fail(PA_ERR_INVALID, "q_out overlaps k or v");
    }
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.tokens = num_tokens;
    p.positions = positions;
    p.slots = slot_mapping;
    p.turns = turns;
    p.num_blocks = num_blocks;
    p.s_block = stride_block;
    p.s_head = stride_head;
    p.s_token = stride_token;
    p.nq = num_q_heads;
    p.nk = p.nv = num_kv_heads;
    p.head_dim = head_dim;
    p.pairs = rotary_dim / 2;
    p.factor = attention_factor;
    p.k_by = quotient_by(k_scale);
    p.v_by = quotient_by(v_scale);
    rc = api_status_ptr(&p.status);
    if (rc) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kv_dtype == PA_KV_FP8_E4M3 ? launch_rope<kAppendFp8>(p, interleaved != 0, s)
                                                     : launch_rope<kAppend>(p, interleaved != 0, s);
    return e == cudaSuccess ? PA_OK : api_cuda_fail(e, "rope_append launch");
}
