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
// Bound by memory: 2 bytes read and 2 written for each channel, a sincos per pair and token.  A CTA serves
// one token: its threads send for the rows first, work out the token's cos and sin meanwhile (one pair
// each, shared through shared memory by all heads), then turn and store.  A thread's unit is 16 channels:
// two 16-byte vectors of the pairs 8 u .. 8 u + 7, so that a thread keeps its eight cos and sin for every
// head it serves.
#include <cmath>
#include <cstring>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kMaxPairs = 128;

struct Rows {                   // [token][head][head_dim] by element strides
    const void *base;
    int64_t token, head;
};

struct RopeParams {
    Rows q, k, v, q_out, k_out;          // v: append only; k_out: pa_rope only
    uint8_t *k_cache, *v_cache;
    const int64_t *positions, *slots;
    const uint64_t *turns;
    int64_t num_blocks, s_block, s_head, s_token;
    int nq, nk, nv, head_dim, pairs, inverse;
    float factor, k_scale, v_scale;
    int *status;
};

enum { kRope = 0, kAppend = 1, kAppendFp8 = 2 };

__device__ __forceinline__ float2 turn_of(uint64_t frequency, int64_t position, bool inverse, float factor) {
    const uint64_t turns = frequency * static_cast<uint64_t>(position);
    const float half_turns = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * factor, (inverse ? -s : s) * factor);
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)   // the first source goes to the upper half
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// E4M3 codes of x / scale: the quotient in fp32, to nearest even, saturated at +-448.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint16_t h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(h[j])
                : "f"(__fdiv_rn(x[4 * i + 2 * j + 1], scale)), "f"(__fdiv_rn(x[4 * i + 2 * j], scale)));
        w[i] = static_cast<uint32_t>(h[0]) | (static_cast<uint32_t>(h[1]) << 16);
    }
    return make_uint2(w[0], w[1]);
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

// Eight results to channel c of head h: a row of q_out or k_out, or of the cache at `at` (element offset
// of the token's slot).
template <int KIND>
__device__ __forceinline__ void put8(const RopeParams &p, int64_t t, int h, int c, int64_t at, const float (&x)[8],
                                     const uint4 &raw, bool turned) {
    if (KIND == kRope || h < p.nq) {
        const __nv_bfloat16 *row = h < p.nq ? row_of(p.q_out, t, h) : row_of(p.k_out, t, h - p.nq);
        *reinterpret_cast<uint4 *>(const_cast<__nv_bfloat16 *>(row) + c) = turned ? pack8(x) : raw;
        return;
    }
    h -= p.nq;
    const bool is_k = h < p.nk;
    uint8_t *pool = is_k ? p.k_cache : p.v_cache;
    const int64_t to = at + (is_k ? h : h - p.nk) * p.s_head + c;
    if (KIND == kAppendFp8)
        *reinterpret_cast<uint2 *>(pool + to) = codes8(x, is_k ? p.k_scale : p.v_scale);
    else
        *reinterpret_cast<uint4 *>(pool + to * 2) = turned ? pack8(x) : raw;
}

// Element offset of a token's slot in the pools; false: the token is skipped (padding, or a slot outside
// the pool, which is flagged).
template <int KIND>
__device__ __forceinline__ bool slot_of(const RopeParams &p, int64_t t, int64_t *at) {
    *at = 0;
    if (KIND == kRope) return true;
    const int64_t slot = p.slots[t];
    if (slot < 0) return false;
    const int64_t page = slot / kBlockSize;
    if (page >= p.num_blocks) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
        return false;
    }
    *at = page * p.s_block + (slot - page * kBlockSize) * p.s_token;
    return true;
}

// Half layout with pairs a multiple of 8, and every interleaved one: 16 channels a unit.
template <int KIND, bool INTERLEAVED>
__global__ void __launch_bounds__(1024) rope_kernel(const __grid_constant__ RopeParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ __align__(16) float2 turns[kMaxPairs];
    const int64_t t = blockIdx.x;
    const int per_head = p.head_dim / 16;            // 4, 8 or 16: blockDim is a multiple of it
    const int u = threadIdx.x & (per_head - 1);
    const int heads = p.nq + p.nk + p.nv;
    const int step = blockDim.x / per_head;
    int h = threadIdx.x / per_head;
    const bool turned = 8 * u < p.pairs;
    // the unit's two vectors
    const int c0 = INTERLEAVED || !turned ? 16 * u : 8 * u;
    const int c1 = INTERLEAVED || !turned ? 16 * u + 8 : p.pairs + 8 * u;
    uint4 a, b;
    if (h < heads) {
        const __nv_bfloat16 *from = source<KIND>(p, t, h);
        a = *reinterpret_cast<const uint4 *>(from + c0);
        b = *reinterpret_cast<const uint4 *>(from + c1);
    }
    int64_t at;
    if (!slot_of<KIND>(p, t, &at)) return;           // the whole CTA
    const int64_t position = p.positions[t];
    for (int i = threadIdx.x; i < p.pairs; i += blockDim.x)
        turns[i] = turn_of(p.turns[i], position, p.inverse != 0, p.factor);
    __syncthreads();
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (8 * u + i < p.pairs) cs[i] = turns[8 * u + i];
    for (; h < heads; h += step) {
        const bool turn = turned && (KIND == kRope || h < p.nq + p.nk);
        float x[8], y[8];
        unpack8(a, x);
        unpack8(b, y);
        if (turn) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (8 * u + i >= p.pairs) continue;
                // pair i of the unit: (x[i], y[i]), or two neighbours of x or y
                float &r0 = !INTERLEAVED ? x[i] : i < 4 ? x[2 * i] : y[2 * i - 8];
                float &r1 = !INTERLEAVED ? y[i] : i < 4 ? x[2 * i + 1] : y[2 * i - 7];
                const float lo = r0, hi = r1;
                r0 = __fmaf_rn(lo, cs[i].x, -hi * cs[i].y);
                r1 = __fmaf_rn(hi, cs[i].x, lo * cs[i].y);
            }
        }
        // values are rotated by their thread's u like the rest, but not turned
        put8<KIND>(p, t, h, c0, at, x, a, turn);
        put8<KIND>(p, t, h, c1, at, y, b, turn);
        if (h + step < heads) {
            const __nv_bfloat16 *from = source<KIND>(p, t, h + step);
            a = *reinterpret_cast<const uint4 *>(from + c0);
            b = *reinterpret_cast<const uint4 *>(from + c1);
        }
    }
}

// Half layout with any other number of pairs: the second halves of the pairs start at any channel, so a
// thread turns a pair, or passes a channel on, at a time.
template <int KIND>
__global__ void __launch_bounds__(256) rope_pairs_kernel(const __grid_constant__ RopeParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float2 turns[kMaxPairs];
    const int64_t t = blockIdx.x;
    int64_t at;
    if (!slot_of<KIND>(p, t, &at)) return;
    const int64_t position = p.positions[t];
    for (int i = threadIdx.x; i < p.pairs; i += blockDim.x)
        turns[i] = turn_of(p.turns[i], position, p.inverse != 0, p.factor);
    __syncthreads();
    auto put = [&](int h, int c, float x) {
        if (KIND == kRope || h < p.nq) {
            const __nv_bfloat16 *row = h < p.nq ? row_of(p.q_out, t, h) : row_of(p.k_out, t, h - p.nq);
            const_cast<__nv_bfloat16 *>(row)[c] = __float2bfloat16_rn(x);
            return;
        }
        h -= p.nq;
        const bool is_k = h < p.nk;
        uint8_t *pool = is_k ? p.k_cache : p.v_cache;
        const int64_t to = at + (is_k ? h : h - p.nk) * p.s_head + c;
        if (KIND == kAppendFp8) {
            uint16_t code;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(code)
                : "f"(0.f), "f"(__fdiv_rn(x, is_k ? p.k_scale : p.v_scale)));
            pool[to] = static_cast<uint8_t>(code);
        } else {
            reinterpret_cast<__nv_bfloat16 *>(pool)[to] = __float2bfloat16_rn(x);
        }
    };
    const int items = p.head_dim - p.pairs;          // pairs, then the channels behind them
    const int turning = (p.nq + p.nk) * items;
    for (int i = threadIdx.x; i < turning; i += blockDim.x) {
        const int h = i / items, c = i - h * items;
        const __nv_bfloat16 *from = source<KIND>(p, t, h);
        if (c < p.pairs) {
            const float lo = __bfloat162float(from[c]), hi = __bfloat162float(from[c + p.pairs]);
            const float2 w = turns[c];
            put(h, c, __fmaf_rn(lo, w.x, -hi * w.y));
            put(h, c + p.pairs, __fmaf_rn(hi, w.x, lo * w.y));
        } else {
            put(h, c + p.pairs, __bfloat162float(from[c + p.pairs]));
        }
    }
    for (int i = threadIdx.x; i < p.nv * p.head_dim; i += blockDim.x) {
        const int h = p.nq + p.nk + i / p.head_dim, c = i & (p.head_dim - 1);
        put(h, c, __bfloat162float(source<KIND>(p, t, h)[c]));
    }
}

template <int KIND>
cudaError_t launch_rope(const RopeParams &p, int64_t tokens, bool interleaved, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(tokens));
    if (!interleaved && p.pairs % 8) return launch_after(rope_pairs_kernel<KIND>, grid, 256, p, stream);
    const int units = (p.nq + p.nk + p.nv) * (p.head_dim / 16);
    int threads = (units + 31) / 32 * 32;
    if (threads > 512) threads = 512;
    return interleaved ? launch_after(rope_kernel<KIND, true>, grid, threads, p, stream)
                       : launch_after(rope_kernel<KIND, false>, grid, threads, p, stream);
}

// ---- argument checks --------------------------------------------------------------------

// The elements of a [tokens][heads][head_dim] tensor in two levels: `outer` steps of runs that span
// `span` elements.  The stride of an axis of length 1 counts as none.
struct Extent {
    uintptr_t at;
    int64_t outer, count, span;     // bytes but for count
};

Extent extent_of(const Rows &r, int64_t tokens, int heads, int head_dim) {
    const int64_t st = tokens > 1 ? r.token : 0, sh = heads > 1 ? r.head : 0;
    const bool by_token = st >= sh;
    Extent e;
    e.at = reinterpret_cast<uintptr_t>(r.base);
    e.outer = 2 * (by_token ? st : sh);
    e.count = by_token ? tokens : heads;
    e.span = 2 * ((by_token ? (heads - 1) * sh : (tokens - 1) * st) + head_dim);
    return e;
}

// False where the two are seen to share no element: apart as a whole, or with the same outer stride and
// runs beside one another (the slices of one projection's rows).
bool may_overlap(const Extent &a, const Extent &b) {
    const uintptr_t a_end = a.at + (a.count - 1) * a.outer + a.span, b_end = b.at + (b.count - 1) * b.outer + b.span;
    if (a_end <= b.at || b_end <= a.at) return false;
    if (a.outer != b.outer || a.outer == 0) return true;
    const int64_t s = a.outer;
    const int64_t d = static_cast<int64_t>(b.at >= a.at ? (b.at - a.at) % s : (s - (a.at - b.at) % s) % s);
    return !(d >= a.span && d + b.span <= s);
}

int check_rows(const char *name, const Rows &r, int64_t tokens, int heads, int head_dim, bool written) {
    if (!r.base || (reinterpret_cast<uintptr_t>(r.base) & 15u))
        return api_fail(PA_ERR_INVALID, "%s is NULL or not 16-byte aligned", name);
    const int64_t st = tokens > 1 ? r.token : 0, sh = heads > 1 ? r.head : 0;
    constexpr int64_t kMost = INT64_C(1) << 40;      // far beyond memory: offsets stay within 64 bits
    if (st < 0 || sh < 0 || st % 8 || sh % 8 || st > kMost || sh > kMost)
        return api_fail(PA_ERR_INVALID, "%s: strides (%lld, %lld) must be multiples of 16 bytes, not negative", name,
                        static_cast<long long>(r.token), static_cast<long long>(r.head));
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
    if (num_tokens > INT32_MAX)
        return api_fail(PA_ERR_UNSUPPORTED, "num_tokens %lld > 2^31 - 1", static_cast<long long>(num_tokens));
    if (nq < 0 || nk < 0) return api_fail(PA_ERR_INVALID, "head counts (%d, %d)", nq, nk);
    if (nq > 65536 || nk > 65536) return api_fail(PA_ERR_UNSUPPORTED, "head counts (%d, %d) > 65536", nq, nk);
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return api_fail(PA_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", head_dim);
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim)
        return api_fail(PA_ERR_INVALID, "rotary_dim %d must be even, from 2 to head_dim %d", rotary_dim, head_dim);
    if (!std::isfinite(factor)) return api_fail(PA_ERR_INVALID, "attention_factor %g", static_cast<double>(factor));
    return PA_OK;
}

// Number of a pair that makes `turns` full turns within `len` positions, as a real number.
double pair_of_turns(double turns, int rotary_dim, double base, double len) {
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    return rotary_dim * std::log(len / (turns * kTwoPi)) / (2 * std::log(base));
}

}  // namespace
}  // namespace pa

extern "C" int pa_rope_table_of(uint64_t *turns_h, const double *frequencies_h, int num_pairs) {
    using namespace pa;
    if (num_pairs < 1 || num_pairs > kMaxPairs)
        return api_fail(PA_ERR_INVALID, "num_pairs %d not in [1, %d]", num_pairs, kMaxPairs);
    if (!turns_h || !frequencies_h) return api_fail(PA_ERR_INVALID, "null pointer argument");
    for (int i = 0; i < num_pairs; ++i)
        if (!std::isfinite(frequencies_h[i])) return api_fail(PA_ERR_INVALID, "frequency %d is not finite", i);
    for (int i = 0; i < num_pairs; ++i) {
        constexpr double kTwoPi = 6.283185307179586476925286766559;
        const double turns = std::fabs(frequencies_h[i]) / kTwoPi;
        const uint64_t part = static_cast<uint64_t>(std::nearbyint(std::ldexp(turns - std::floor(turns), 64)));
        turns_h[i] = frequencies_h[i] < 0 ? 0 - part : part;
    }
    return PA_OK;
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
    double f[kMaxPairs];
    const double b = scaling == PA_ROPE_NTK ? base * std::pow(factor, rotary_dim / (rotary_dim - 2.0)) : base;
    for (int i = 0; i < n; ++i) f[i] = std::pow(b, -2.0 * i / rotary_dim);
    float m = 1.f;
    if (scaling == PA_ROPE_LINEAR) {
        for (int i = 0; i < n; ++i) f[i] /= factor;
    } else if (scaling == PA_ROPE_BANDS) {
        for (int i = 0; i < n; ++i) {
            const double turns = len * f[i] / 6.283185307179586476925286766559;
            const double s = std::fmin(std::fmax((turns - low) / (high - low), 0.0), 1.0);
            f[i] *= (1 - s) / factor + s;
        }
    } else if (scaling == PA_ROPE_YARN) {
        const double first = std::fmax(std::floor(pair_of_turns(high, rotary_dim, base, len)), 0.0);
        const double last = std::fmin(std::ceil(pair_of_turns(low, rotary_dim, base, len)), rotary_dim - 1.0);
        for (int i = 0; i < n; ++i) {
            const double s = std::fmin(std::fmax((i - first) / std::fmax(last - first, 0.001), 0.0), 1.0);
            f[i] *= s / factor + (1 - s);
        }
        if (factor > 1) m = static_cast<float>(0.1 * std::log(factor) + 1);
    }
    const int rc = pa_rope_table_of(turns_h, f, n);
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
    p.positions = positions;
    p.turns = turns;
    p.nq = num_q_heads;
    p.nk = num_k_heads;
    p.head_dim = head_dim;
    p.pairs = rotary_dim / 2;
    p.inverse = inverse ? 1 : 0;
    p.factor = attention_factor;
    const cudaError_t e = launch_rope<kRope>(p, num_tokens, interleaved != 0, static_cast<cudaStream_t>(stream));
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
    if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 15u)
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
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    rc = api_status_ptr(&p.status);
    if (rc) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kv_dtype == PA_KV_FP8_E4M3 ? launch_rope<kAppendFp8>(p, num_tokens, interleaved != 0, s)
                                                     : launch_rope<kAppend>(p, num_tokens, interleaved != 0, s);
    return e == cudaSuccess ? PA_OK : api_cuda_fail(e, "rope_append launch");
}
