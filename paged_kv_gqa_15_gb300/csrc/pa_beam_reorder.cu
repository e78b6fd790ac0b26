// pa_beam_reorder.cu -- the paged cache follows the chosen beams: beam slot j goes on from what its parent
// slot held.
//
// Full pages never change again, so they are shared: slot j's block-table row takes its parent's page ids.
// Only the page that the next tokens go to is a slot's own, and its rows so far are copied, in every pool.
//
// Both are permutations in place, a slot being the parent of some while it takes over another.  One thread
// takes one 16-byte chunk of one row of the page, for all slots of a request (or one column of their tables):
// it reads what every moving slot needs, then writes.  Nobody else touches these chunks: no barrier, no second
// buffer.
//
// Bound by memory for many layers (each moved row is read and written once), by the chain lengths -> page
// ids -> rows for few.  So a CTA goes through that chain once for several pools where there
// are many, and only over the rows that there are.  32 layers, 32 requests of 4 beams, 8 heads of 128
// channels: 179 MB in 30 us, 88 % of the copy rate; 2 pools of one request 3.1 us.
#include <cstring>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kMaxPools = 128;       // pools per launch
constexpr int kThreads = 256;

struct ReorderParams {
    uint8_t *pools[kMaxPools];
    int32_t *block_tables;
    const int32_t *seq_lens, *parents;
    int64_t num_blocks, b_block, b_head, b_token;   // strides in bytes
    int num_pools, num_beams, num_kv_heads, max_blocks;
    int chunk_bits;                                 // a row's chunks: 1 << chunk_bits
    int pools_per_cta, copy_ctas;                   // copy_ctas of a request; one more moves its tables
    int *status;
};

// Grid: x = shares of the pools, then the tables; y = request.  BEAMS: an upper bound of num_beams.
template <int BEAMS>
__global__ void __launch_bounds__(kThreads) reorder_kernel(const __grid_constant__ ReorderParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ int parent[BEAMS], page[BEAMS], len[BEAMS];
    __shared__ bool searched[BEAMS];                // in the search: its page is its own
    const int tid = threadIdx.x, n = p.num_beams;
    const int64_t slot0 = static_cast<int64_t>(blockIdx.y) * n;
    int32_t *tables = p.block_tables + slot0 * p.max_blocks;
    const bool tables_cta = static_cast<int>(blockIdx.x) == p.copy_ctas;
    if (tid < n) {
        const int L = p.seq_lens[slot0 + tid];
        len[tid] = L;
        searched[tid] = p.parents[slot0 + tid] >= 0;
        page[tid] = -1;
        if (L >= 0 && L / kBlockSize < p.max_blocks) {
            const int id = tables[static_cast<int64_t>(tid) * p.max_blocks + L / kBlockSize];
            if (L % kBlockSize && id >= 0 && id < p.num_blocks) page[tid] = id;
        }
    }
    __syncthreads();
    // a slot that cannot move is its own parent
    bool moves = false;
    if (tid < n) {
        const int L = len[tid], from = p.parents[slot0 + tid];
        bool bad = from < -1 || from >= n;
        if (!bad && from >= 0 && from != tid) {
            bad = L < 0 || L > p.max_blocks * kBlockSize || len[from] != L;
            if (!bad && L % kBlockSize) {
                bad = page[tid] < 0 || page[from] < 0;
                for (int i = 0; i < n; ++i) bad |= i != tid && searched[i] && page[i] == page[tid];
            }
            moves = !bad;
        }
        parent[tid] = moves ? from : tid;
        if (bad && tables_cta) atomicOr(p.status, kStatusBounds);
    }
    if (!__syncthreads_or(moves)) return;
    if (tables_cta) {
        int most = 0;
        for (int j = 0; j < n; ++j)
            if (parent[j] != j) most = max(most, len[j] / kBlockSize);
        for (int c = tid; c < most; c += kThreads) {
            int32_t id[BEAMS];
#pragma unroll
            for (int j = 0; j < BEAMS; ++j)
                if (j < n && parent[j] != j && c < len[j] / kBlockSize)
                    id[j] = tables[static_cast<int64_t>(parent[j]) * p.max_blocks + c];
#pragma unroll
            for (int j = 0; j < BEAMS; ++j)
                if (j < n && parent[j] != j && c < len[j] / kBlockSize)
                    tables[static_cast<int64_t>(j) * p.max_blocks + c] = id[j];
        }
        return;
    }
    int rows = 0;
    for (int j = 0; j < n; ++j)
        if (parent[j] != j) rows = max(rows, len[j] % kBlockSize);
    const int items = (p.num_kv_heads * rows) << p.chunk_bits;
    const int pool0 = blockIdx.x * p.pools_per_cta, pool1 = min(p.num_pools, pool0 + p.pools_per_cta);
    constexpr int kAhead = BEAMS <= 4 ? 2 : 1;      // chunks of a thread that are read before any is written
    for (int pool = pool0; pool < pool1; ++pool)
        for (int i0 = tid; i0 < items; i0 += kAhead * kThreads) {
            uint4 v[kAhead][BEAMS];
            uint8_t *at[kAhead];
            int row[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int i = i0 + a * kThreads;
                const int r = i >> p.chunk_bits, h = r / rows;
                row[a] = i < items ? r - h * rows : kBlockSize;
                at[a] = p.pools[pool] + h * p.b_head + row[a] * p.b_token + (i & ((1 << p.chunk_bits) - 1)) * 16;
#pragma unroll
                for (int j = 0; j < BEAMS; ++j)
                    if (j < n && parent[j] != j && row[a] < len[j] % kBlockSize)
                        v[a][j] = *reinterpret_cast<const uint4 *>(at[a] + page[parent[j]] * p.b_block);
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
#pragma unroll
                for (int j = 0; j < BEAMS; ++j)
                    if (j < n && parent[j] != j && row[a] < len[j] % kBlockSize)
                        *reinterpret_cast<uint4 *>(at[a] + page[j] * p.b_block) = v[a][j];
        }
}

}  // namespace
}  // namespace pa

extern "C" int pa_beam_reorder(void *const *pools, int num_pools, int32_t *block_tables, const int32_t *seq_lens,
                               const int32_t *parents, int num_requests, int num_beams, int num_kv_heads,
                               int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
                               int64_t stride_block, int64_t stride_head, int64_t stride_token, int kv_dtype,
                               void *stream) {
    using namespace pa;
    if (num_pools < 0 || num_requests < 0)
        return api_fail(PA_ERR_INVALID, "num_pools %d, num_requests %d", num_pools, num_requests);
    if (num_beams <= 0) return api_fail(PA_ERR_INVALID, "num_beams %d", num_beams);
    if (num_beams > PA_MAX_BEAMS) return api_fail(PA_ERR_UNSUPPORTED, "num_beams %d > %d", num_beams, PA_MAX_BEAMS);
    int rc = api_check_heads(head_dim, num_kv_heads, num_kv_heads);
    if (rc) return rc;
    rc = api_check_kv_dtype(kv_dtype, 1.f, 1.f);
    if (rc) return rc;
    rc = api_check_pool(head_dim, block_size, num_blocks, num_kv_heads, stride_block, stride_head, stride_token,
                        kv_dtype);
    if (rc) return rc;
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > INT32_MAX / kBlockSize)
        return api_fail(PA_ERR_INVALID, "max_blocks_per_seq %d", max_blocks_per_seq);
    if (num_requests > 65535) return api_fail(PA_ERR_UNSUPPORTED, "num_requests %d > 65535", num_requests);
    if (num_kv_heads > 65536) return api_fail(PA_ERR_UNSUPPORTED, "num_kv_heads %d > 65536", num_kv_heads);
    if (num_requests == 0) return PA_OK;
    if (!block_tables || !seq_lens || !parents || (num_pools > 0 && !pools))
        return api_fail(PA_ERR_INVALID, "null pointer argument");
    if (!api_aligned(block_tables, 4) || !api_aligned(seq_lens, 4) || !api_aligned(parents, 4))
        return api_fail(PA_ERR_INVALID, "block_tables, seq_lens and parents must be 4-byte aligned");
    const int64_t slots = static_cast<int64_t>(num_requests) * num_beams;
    if (api_overlap(block_tables, slots * max_blocks_per_seq, seq_lens, slots) ||
        api_overlap(block_tables, slots * max_blocks_per_seq, parents, slots))
        return api_fail(PA_ERR_INVALID, "block_tables must not overlap seq_lens or parents");
    for (int i = 0; i < num_pools; ++i)
        if (!pools[i] || !api_aligned(pools[i], 16))
            return api_fail(PA_ERR_INVALID, "pools[%d] is NULL or not 16-byte aligned", i);
    // a pool listed twice would have its rows moved by two threads at once
    for (int i = 1; i < num_pools; ++i)
        for (int j = 0; j < i; ++j)
            if (pools[j] == pools[i]) return api_fail(PA_ERR_INVALID, "pools[%d] is listed twice", i);
    ReorderParams p;
    std::memset(&p, 0, sizeof p);
    const int elem = kv_dtype == PA_KV_FP8_E4M3 ? 1 : 2;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.parents = parents;
    p.num_blocks = num_blocks;
    p.b_block = stride_block * elem;
    p.b_head = stride_head * elem;
    p.b_token = stride_token * elem;
    p.num_beams = num_beams;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    for (int chunks = head_dim * elem / 16; chunks > 1; chunks /= 2) ++p.chunk_bits;
    rc = api_status_ptr(&p.status);
    if (rc) return rc;
    for (int at = 0; at == 0 || at < num_pools; at += kMaxPools) {
        p.num_pools = num_pools - at < kMaxPools ? num_pools - at : kMaxPools;
        for (int i = 0; i < p.num_pools; ++i) p.pools[i] = static_cast<uint8_t *>(pools[at + i]);
        // enough CTAs to even out requests of more and fewer rows: two waves of eight an SM
        const int64_t share = (static_cast<int64_t>(p.num_pools) * num_requests + 152 * 16 - 1) / (152 * 16);
        p.pools_per_cta = static_cast<int>(share < p.num_pools ? share : p.num_pools);
        p.copy_ctas = p.num_pools ? (p.num_pools + p.pools_per_cta - 1) / p.pools_per_cta : 0;
        // the tables move with the first launch
        const dim3 grid(static_cast<unsigned>(p.copy_ctas + (at == 0)), static_cast<unsigned>(num_requests));
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        const cudaError_t e = num_beams <= 4    ? launch_after(reorder_kernel<4>, grid, kThreads, p, s)
                              : num_beams <= 8  ? launch_after(reorder_kernel<8>, grid, kThreads, p, s)
                              : num_beams <= 16 ? launch_after(reorder_kernel<16>, grid, kThreads, p, s)
                                                : launch_after(reorder_kernel<32>, grid, kThreads, p, s);
        if (e != cudaSuccess) return api_cuda_fail(e, "reorder_kernel launch");
    }
    return PA_OK;
}
