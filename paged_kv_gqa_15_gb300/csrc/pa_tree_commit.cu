// pa_tree_commit.cu -- the accepted path of a drafted token tree becomes the sequence's
// next tokens: in every pool, token C + i takes the row of token C + a_i.
//
// One thread owns one 16-byte chunk of a (sequence, pool, kv head)'s rows and walks the
// path in order.  The path ascends, so a_i >= i and a row is overwritten only after every
// step that reads it (row i is read by steps i' <= i alone): no other thread touches the
// chunk's column, so the move is safe in place without any barrier.
//
// Bound by latency: lengths, path, page ids and rows are four dependent reads, and a step moves
// little (31 MB read and written for 118 accepted nodes in 32 layers: 9.4 us, 4.6 at the copy
// rate).  Hence a thread per chunk, all pools in one launch, and four steps' rows read at once.
#include <cstring>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kMaxPools = 128;   // pools per launch
constexpr int kThreads = 128;
constexpr int kAhead = 4;        // path steps whose rows are read before any is written

struct CommitParams {
    uint8_t *pools[kMaxPools];
    const int32_t *block_tables, *seq_lens, *qo_indptr, *accepted, *accept_lens;
    int32_t *new_seq_lens;
    int64_t num_blocks, b_block, b_head, b_token;   // strides in bytes
    int num_pools, max_tree_len, max_accept, num_kv_heads, max_blocks, chunks;
    int write_lens;                                 // this launch writes new_seq_lens
    int *status;
};

// Grid: x = (pool, kv head, chunk) threads, y = sequence.
__global__ void __launch_bounds__(kThreads) commit_kernel(const __grid_constant__ CommitParams p) {
    const int b = blockIdx.y;
    const int t = blockIdx.x * kThreads + threadIdx.x;
    const bool first = t == 0;
    const int T = p.qo_indptr[b + 1] - p.qo_indptr[b];
    const int L = p.seq_lens[b];
    const int n_in = p.accept_lens[b];
    if (T < 0 || T > p.max_tree_len || L < T || L > p.max_blocks * kBlockSize) {
        if (first) {
            atomicOr(p.status, kStatusBounds);
            if (p.write_lens) p.new_seq_lens[b] = L;
        }
        return;
    }
    const int C = L - T;
    // the path up to its first entry that is out of range or does not ascend
    const int32_t *path = p.accepted + static_cast<int64_t>(b) * p.max_accept;
    const int most = min(max(n_in, 0), p.max_accept);
    int n = 0;
    for (int last = -1; n < most; ++n) {
        const int a = path[n];
        if (a <= last || a >= T) break;
        last = a;
    }
    if (first) {
        if (n != n_in) atomicOr(p.status, kStatusBounds);
        if (p.write_lens) p.new_seq_lens[b] = C + n;
    }
    if (t >= p.num_pools * p.num_kv_heads * p.chunks) return;
    const int c = t % p.chunks;
    const int h = t / p.chunks % p.num_kv_heads;
    uint8_t *base = p.pools[t / p.chunks / p.num_kv_heads] + h * p.b_head + c * 16;
    const int32_t *bt = p.block_tables + static_cast<int64_t>(b) * p.max_blocks;
    auto place = [&](int tok) -> uint8_t * {
        const int page = bt[tok / kBlockSize];
        if (page < 0 || page >= p.num_blocks) return nullptr;
        return base + page * p.b_block + (tok % kBlockSize) * p.b_token;
    };
    bool bad = false;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        uint4 v[kAhead];
        uint8_t *to[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            to[u] = nullptr;
            const int i = i0 + u;
            if (i >= n || path[i] == i) continue;    // a node already in place
            const uint8_t *from = place(C + path[i]);
            to[u] = place(C + i);
            if (from && to[u]) {
                v[u] = *reinterpret_cast<const uint4 *>(from);
            } else {
                bad = true;
                to[u] = nullptr;
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (to[u]) *reinterpret_cast<uint4 *>(to[u]) = v[u];
    }
    if (bad) atomicOr(p.status, kStatusBounds);
}

}  // namespace
}  // namespace pa

extern "C" int pa_tree_commit(void *const *pools, int num_pools, const int32_t *block_tables,
                              const int32_t *seq_lens, const int32_t *qo_indptr,
                              const int32_t *accepted, const int32_t *accept_lens,
                              int32_t *new_seq_lens, int num_seqs, int max_tree_len,
                              int max_accept, int num_kv_heads, int head_dim, int block_size,
                              int max_blocks_per_seq, int64_t num_blocks, int64_t stride_block,
                              int64_t stride_head, int64_t stride_token, int kv_dtype,
                              void *stream) {
    using namespace pa;
    if (num_pools < 0 || num_seqs < 0)
        return api_fail(PA_ERR_INVALID, "num_pools %d, num_seqs %d", num_pools, num_seqs);
    int rc = api_check_heads(head_dim, num_kv_heads, num_kv_heads);
    if (rc) return rc;
    rc = api_check_kv_dtype(kv_dtype, 1.f, 1.f);
    if (rc) return rc;
    rc = api_check_pool(head_dim, block_size, num_blocks, num_kv_heads, stride_block, stride_head,
                        stride_token, kv_dtype);
    if (rc) return rc;
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > INT32_MAX / kBlockSize)
        return api_fail(PA_ERR_INVALID, "max_blocks_per_seq %d", max_blocks_per_seq);
    if (max_tree_len < 0 || max_accept < 0)
        return api_fail(PA_ERR_INVALID, "max_tree_len %d, max_accept %d", max_tree_len, max_accept);
    if (num_seqs > 65535) return api_fail(PA_ERR_UNSUPPORTED, "num_seqs %d > 65535", num_seqs);
    if (num_kv_heads > (1 << 16))
        return api_fail(PA_ERR_UNSUPPORTED, "num_kv_heads %d > 65536", num_kv_heads);
    if (num_seqs == 0) return PA_OK;
    if (!block_tables || !seq_lens || !qo_indptr || !accept_lens || !new_seq_lens ||
        (max_accept > 0 && !accepted) || (num_pools > 0 && !pools))
        return api_fail(PA_ERR_INVALID, "null pointer argument");
    if (api_overlap(new_seq_lens, num_seqs, seq_lens, num_seqs) ||
        api_overlap(new_seq_lens, num_seqs, accept_lens, num_seqs) ||
        api_overlap(new_seq_lens, num_seqs, qo_indptr, num_seqs + 1) ||
        api_overlap(new_seq_lens, num_seqs, accepted, static_cast<int64_t>(num_seqs) * max_accept) ||
        api_overlap(new_seq_lens, num_seqs, block_tables, static_cast<int64_t>(num_seqs) * max_blocks_per_seq))
        return api_fail(PA_ERR_INVALID, "new_seq_lens must not overlap what the call reads");
    for (int i = 0; i < num_pools; ++i)
        if (!pools[i] || (reinterpret_cast<uintptr_t>(pools[i]) & 15u))
            return api_fail(PA_ERR_INVALID, "pools[%d] is NULL or not 16-byte aligned", i);
    // a pool moved twice would take its rows from where the first move left others
    for (int i = 1; i < num_pools; ++i) {
        bool again = false;
        for (int j = 0; j < i; ++j) again |= pools[j] == pools[i];
        if (again) return api_fail(PA_ERR_INVALID, "pools[%d] is listed twice", i);
    }
    CommitParams p;
    std::memset(&p, 0, sizeof p);
    const int elem = kv_dtype == PA_KV_FP8_E4M3 ? 1 : 2;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.qo_indptr = qo_indptr;
    p.accepted = accepted;
    p.accept_lens = accept_lens;
    p.new_seq_lens = new_seq_lens;
    p.num_blocks = num_blocks;
    p.b_block = stride_block * elem;
    p.b_head = stride_head * elem;
    p.b_token = stride_token * elem;
    p.max_tree_len = max_tree_len;
    p.max_accept = max_accept;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.chunks = head_dim * elem / 16;
    rc = api_status_ptr(&p.status);
    if (rc) return rc;
    for (int at = 0; at == 0 || at < num_pools; at += kMaxPools) {
        p.num_pools = num_pools - at < kMaxPools ? num_pools - at : kMaxPools;
        p.write_lens = at == 0;
        for (int i = 0; i < p.num_pools; ++i) p.pools[i] = static_cast<uint8_t *>(pools[at + i]);
        const int64_t threads = static_cast<int64_t>(p.num_pools) * num_kv_heads * p.chunks;
        const dim3 grid(static_cast<unsigned>(threads > 0 ? (threads + kThreads - 1) / kThreads : 1),
                        static_cast<unsigned>(num_seqs));
        commit_kernel<<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return api_cuda_fail(e, "commit_kernel launch");
    }
    return PA_OK;
}
