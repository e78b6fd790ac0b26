// pa_tree.cu -- attention of drafted token trees over the paged cache.
//
// What it computes: sequence b's cache ends in its T drafted nodes (the last T of its L
// tokens); row i of the tree and query head h attend to the C = L - T context tokens
// (under a sliding window, those from C + n_i - window on, n_i the nodes the row sees) and
// to the nodes named by the row's bit mask; softmax(sm_scale q . k) weighted sum of v.
//
// One warp per (row, query head): lanes own head_dim / 32 channels each, keys are taken one
// at a time with the running maximum and sum of an online softmax in fp32.
#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// Sequence b's drafted rows and lengths; ok is false (and the device status flagged by
// `flag`) when its rows or lengths make no sense.
struct TreeSeq {
    int row0, T, L;
    bool ok;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int b, bool flag) {
    TreeSeq s;
    s.row0 = p.qo_indptr[b];
    const int row1 = p.qo_indptr[b + 1];
    s.T = row1 - s.row0;
    s.L = max(p.seq_lens[b], 0);
    const int cap = p.max_blocks * kBlockSize;
    bool bad = false;
    if (s.L > cap) {
        s.L = cap;
        bad = true;
    }
    s.ok = s.row0 >= 0 && row1 >= s.row0 && row1 <= p.total_rows && s.T <= p.max_tree_len &&
           s.T <= s.L;
    if (flag && (bad || !s.ok)) atomicOr(p.status, kStatusBounds);
    if (!s.ok) s.T = 0;
    return s;
}

template <int HD, bool FP8>
__global__ void __launch_bounds__(128) tree_kernel(const __grid_constant__ TreeParams p) {
    constexpr int D = HD / 32;
    const int b = blockIdx.z, i = blockIdx.x, lane = threadIdx.x & 31;
    const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
    const TreeSeq s = tree_seq(p, b, i == 0 && blockIdx.y == 0 && threadIdx.x == 0);
    if (i >= s.T || h >= p.num_q_heads) return;
    const int kh = h / (p.num_q_heads / p.num_kv_heads);
    const int64_t row = s.row0 + i;
    const uint64_t *mask = p.tree_mask + row * p.mask_words;
    const int C = s.L - s.T;
    int lo = 0;
    if (p.window > 0) {
        int n = 0;
        for (int w = 0; w * 64 < s.T; ++w) {
            const int left = s.T - w * 64;
            n += __popcll(left >= 64 ? mask[w] : mask[w] & ((1ull << left) - 1));
        }
        lo = max(0, min(C, C + n - p.window));
    }
    float q[D], acc[D], m = -INFINITY, l = 0.f;
    const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(p.q) + (row * p.num_q_heads + h) * HD;
    for (int d = 0; d < D; ++d) {
        q[d] = __bfloat162float(qr[lane * D + d]) * p.scale_log2 * p.k_scale;
        acc[d] = 0.f;
    }
    const int32_t *bt = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
    for (int j = lo; j < s.L; ++j) {
        if (j >= C && !((mask[(j - C) >> 6] >> ((j - C) & 63)) & 1)) continue;
        const int page = bt[j / kBlockSize];
        if (page < 0 || page >= p.num_blocks) {
            if (lane == 0) atomicOr(p.status, kStatusBounds);
            continue;
        }
        const int64_t off = page * p.s_block + kh * p.s_head + (j % kBlockSize) * p.s_token + lane * D;
        float k[D], v[D];
        for (int d = 0; d < D; ++d) {
            if constexpr (FP8) {
                k[d] = e4m3x2_to_float2(static_cast<const uint8_t *>(p.k_cache)[off + d]).x;
                v[d] = e4m3x2_to_float2(static_cast<const uint8_t *>(p.v_cache)[off + d]).x;
            } else {
                k[d] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.k_cache)[off + d]);
                v[d] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.v_cache)[off + d]);
            }
        }
        float x = 0.f;
        for (int d = 0; d < D; ++d) x = fmaf(q[d], k[d], x);
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
        const float mn = fmaxf(m, x);
        const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float e = x == -INFINITY ? 0.f : exp2f(x - mn);
        l = l * f + e;
        for (int d = 0; d < D; ++d) acc[d] = acc[d] * f + e * v[d];
        m = mn;
    }
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + (row * p.num_q_heads + h) * HD;
    const float inv = l > 0.f ? p.v_scale / l : 0.f;
    for (int d = 0; d < D; ++d) o[lane * D + d] = __float2bfloat16_rn(acc[d] * inv);
}

template <int HD>
cudaError_t launch_hd(const TreeParams &p, cudaStream_t stream) {
    const dim3 grid(p.max_tree_len, (p.num_q_heads + 3) / 4, p.num_seqs);
    if (p.kv_fp8) tree_kernel<HD, true><<<grid, 128, 0, stream>>>(p);
    else tree_kernel<HD, false><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_decode(const TreeParams &p, int head_dim, cudaStream_t stream) {
    switch (head_dim) {
        case 64: return launch_hd<64>(p, stream);
        case 128: return launch_hd<128>(p, stream);
        case 256: return launch_hd<256>(p, stream);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace pa

extern "C" size_t pa_tree_decode_workspace_size(int num_seqs, int max_tree_len, int num_q_heads,
                                                int num_kv_heads, int head_dim) {
    (void)num_seqs, (void)max_tree_len, (void)num_q_heads, (void)num_kv_heads, (void)head_dim;
    return 256;
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
