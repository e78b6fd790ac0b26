/*
 * pa.h -- C ABI of the paged-KV GQA attention library for GB300 (sm_103a).
 *
 * Operations (each cites the page section that defines it):
 *   pa_write_cache      reshape_and_cache scatter of new K/V rows into pages
 *                       ("paged_attn.py", PagedAttention.write_to_paged_cache)
 *   pa_decode           single-pass paged GQA decode
 *                       ("paged_attn.py", PagedAttention._forward_decode_pytorch
 *                        and the paged_attention_v1 call in forward_decode)
 *   pa_decode_split     split-KV decode: 512-token partitions with fp32
 *                       per-partition max / sum / partial output, then a
 *                       log-sum-exp merge ("paged_attn.py", forward_decode, V2
 *                       branch; "libmir-cuda attention/mod.rs",
 *                       SplitPagedAttention and its workspace); its two halves
 *                       are also exposed as pa_decode_partitions and
 *                       pa_decode_merge, and pa_decode_split_static runs it on a
 *                       library-owned scratch buffer (no caller workspace)
 *   pa_ragged_prefill   ragged (varlen) causal prefill of many requests in one
 *                       launch through qo_indptr / kv_indptr, over contiguous
 *                       or paged K/V ("spark_runtime/flashinfer.rs",
 *                       ragged_prefill_bf16_hd256; "paged_attn.py",
 *                       _forward_prefix_pytorch)
 *   pa_tree_decode      verification of drafted tokens: the nodes of one token
 *                       tree per sequence attend to the sequence's cache and to
 *                       the nodes their tree mask names; pa_tree_commit then
 *                       moves the K/V rows of the accepted path behind the
 *                       context, in every layer (no page defines them)
 *   pa_page_bounds, pa_select_pages, pa_decode_pages  decode over the pages that
 *                       per-page bounds of the keys rank highest for the step's
 *                       query, chosen per sequence and kv head (no page defines
 *                       them)
 *   pa_rope, pa_rope_append  rotary positions of q and k, alone and on k's way into
 *                       the cache; pa_rope_table makes their frequencies (no page
 *                       defines them)
 *   pa_beam_select, pa_beam_reorder  beam search: the best continuations over beams
 *                       and vocabulary, and the cache following the chosen beams (no
 *                       page defines them)
 *   pa_block_table_sync upload of the changed rows of a block table, for
 *                       CUDA-graph replays of the decode ("libmir-cuda
 *                       attention/mod.rs", captured decode nodes)
 *   pa_copy_blocks      copy-on-write page copies inside every layer's K and
 *                       V pools ("paged_attn.py", PagedAttention.copy_blocks)
 *   pa_swap_blocks      page copies between pools on the device and in pinned
 *                       host memory ("paged_attn.py", PagedAttention.swap_blocks)
 *   pa_selftest_wait_timeout  one bounded pipeline wait run out on purpose, to
 *                       check the PA_ERR_TIMEOUT path (no page defines it)
 *
 * The decode entry points take kv_dtype (PA_KV_BF16 or PA_KV_FP8_E4M3) with
 * k_scale / v_scale; pa_write_cache quantises into an FP8 pool with the same
 * arguments ("paged_attn.py", kv_cache_dtype, k_scale and v_scale).
 *
 * Conventions shared by every entry point:
 *  - All data pointers are DEVICE pointers of the current CUDA device unless
 *    the name ends in _h (host).  The caller owns all memory; no entry point
 *    allocates, frees or synchronises (except pa_get_device_status, which
 *    synchronises `stream`).  Work is enqueued on `stream` (a cudaStream_t,
 *    NULL = legacy default stream) and returns immediately.
 *  - bf16 tensors are passed as void pointers to IEEE bfloat16 data.
 *  - KV pools are addressed by element strides (stride_block, stride_head,
 *    stride_token) in elements of the pool's type (bytes for an FP8 pool), each
 *    a multiple of 16 bytes; the head_dim axis is contiguous.  The default layout is
 *    HND per page, [num_blocks][num_kv_heads][block_size][head_dim], i.e.
 *    strides (nkv*bs*hd, bs*hd, hd).  The NHD page layout
 *    [num_blocks][block_size][num_kv_heads][head_dim] is (bs*nkv*hd, hd, nkv*hd).
 *    K and V pools share one set of strides.
 *  - Supported shapes: head_dim in {64, 128, 256}; block_size == 16;
 *    num_q_heads % num_kv_heads == 0, with any group size g = num_q_heads /
 *    num_kv_heads ("paged_attn.py", num_queries_per_kv).  Query head h reads kv
 *    head h / g.  The decode kernels serve some group sizes directly (on the
 *    tensor cores bf16 3-16 at head_dim 128 and 3-8 at head_dim 64, fp8 3-8 at
 *    head_dim 128; the CUDA-core kernel 1, 2, 4 and 8); any other g runs as
 *    several groups of a divisor of g per kv head, each reading that kv head's
 *    pages (through L2).
 *    Pointers must be 16-byte aligned.
 *  - sliding_window (decode and prefill): a query at position pos attends only
 *    to keys j > pos - sliding_window, the sliding_window most recent keys
 *    including its own position ("paged_attn.py", forward_prefix's
 *    sliding_window; "libmir-cuda attention/mod.rs", active_partitions(token
 *    count, window)).  sliding_window <= 0 means no window.  A decode query sits
 *    at position seq_len - 1.  Block-table entries of pages that lie wholly
 *    before a query's window are never read, so a caller may recycle them.
 *  - Return value: PA_OK or an error status; on error nothing was enqueued and
 *    pa_last_error() (thread-local) describes the problem.
 *  - Device-side guards: a block-table entry outside [0, num_blocks), a
 *    seq_len larger than max_blocks_per_seq * block_size, or a slot outside
 *    the pool is never dereferenced: the affected tokens contribute nothing and
 *    a device status word records PA_ERR_DEVICE_BOUNDS.  Every pipeline wait
 *    is bounded; a wait that runs out records PA_ERR_TIMEOUT and the kernel
 *    returns.  A kernel that finds its launch unusable on the device (its
 *    realigned shared-memory tiles not fitting the launch's shared memory) does
 *    no work and records PA_ERR_UNSUPPORTED.  Read (and clear) that word with
 *    pa_get_device_status().
 */
#ifndef PA_H
#define PA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID = 1,       /* bad argument (null pointer, negative size, ...) */
    PA_ERR_UNSUPPORTED = 2,   /* valid but unsupported shape or layout */
    PA_ERR_CUDA = 3,          /* a CUDA runtime call failed */
    PA_ERR_WORKSPACE = 4,     /* workspace too small or misaligned */
    PA_ERR_TIMEOUT = 5,       /* device-side bounded wait ran out */
    PA_ERR_DEVICE_BOUNDS = 6  /* device-side index guard fired */
} pa_status;

/*
 * KV cache element types ("paged_attn.py": kv_cache_dtype, k_scale, v_scale on
 * write_to_paged_cache and forward_decode).  PA_KV_FP8_E4M3 pools hold one byte
 * per element, an OCP FP8 E4M3 code (sign, 4 exponent bits with bias 7, 3
 * mantissa bits, largest finite 448, no infinities): the cache write stores the
 * code nearest to the fp32 quotient x / k_scale (v_scale for V), ties to even,
 * saturating at +-448; the decode reads code value * k_scale (v_scale).  The
 * scales must be positive and finite.  With PA_KV_BF16 they are ignored.
 * Paged prefill reads bf16 pools only.
 */
typedef enum { PA_KV_BF16 = 0, PA_KV_FP8_E4M3 = 1 } pa_kv_dtype;

/* Tokens per split-KV partition ("paged_attn.py", _PARTITION_SIZE). */
#define PA_PARTITION_TOKENS 512

/*
 * pa_write_cache -- reshape_and_cache.
 * For each token t in [0, num_tokens) with slot = slot_mapping[t] >= 0, copies
 * k[t][h][:] into k_cache at page slot / block_size, head h, row
 * slot % block_size (and v likewise): bit for bit into a PA_KV_BF16 pool, or as
 * the E4M3 codes of the elements divided by k_scale (v_scale) into a
 * PA_KV_FP8_E4M3 pool (see pa_kv_dtype).  slot < 0 skips the token
 * (padding).  Slots >= num_blocks * block_size are not written and set
 * PA_ERR_DEVICE_BOUNDS in the device status word.  Two tokens with the same
 * slot in one call give an unspecified winner.
 *   k, v          [num_tokens][num_kv_heads][head_dim] bf16, contiguous
 *   k_cache, v_cache  pools of kv_dtype addressed by the strides (see conventions)
 *   slot_mapping  [num_tokens] int64
 */
int pa_write_cache(const void *k, const void *v, void *k_cache, void *v_cache,
                   const int64_t *slot_mapping, int64_t num_tokens, int num_kv_heads,
                   int head_dim, int block_size, int64_t num_blocks,
                   int64_t stride_block, int64_t stride_head, int64_t stride_token,
                   int kv_dtype, float k_scale, float v_scale, void *stream);

/*
 * pa_decode -- single-pass paged GQA decode (one query token per sequence).
 * For sequence b and query head h (kv head kh = h / (num_q_heads/num_kv_heads)):
 *   out[b][h] = softmax(sm_scale * q[b][h] . K_j) weighted sum of V_j over
 *   j < seq_lens[b], with token j at page block_tables[b][j / block_size],
 *   row j % block_size.  seq_lens[b] == 0 gives a zero row.
 *   out, q        [num_seqs][num_q_heads][head_dim] bf16
 *   block_tables  [num_seqs][max_blocks_per_seq] int32 (entries past
 *                 ceil(seq_len / block_size) are never read)
 *   seq_lens      [num_seqs] int32
 *   k_cache, v_cache, kv_dtype, k_scale, v_scale  the pools and their element
 *                 type (see pa_kv_dtype)
 * One CTA walks the whole sequence of its (b, kv head); suited to short
 * contexts or large batches.  Allocates nothing.
 */
int pa_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
              const int32_t *block_tables, const int32_t *seq_lens, int num_seqs,
              int num_q_heads, int num_kv_heads, int head_dim, int block_size,
              int max_blocks_per_seq, int64_t num_blocks, int64_t stride_block,
              int64_t stride_head, int64_t stride_token, float sm_scale, int sliding_window,
              int kv_dtype, float k_scale, float v_scale, void *stream);

/*
 * Bytes of workspace pa_decode_split needs (256-byte aligned sub-buffers):
 *   P = ceil(max_seq_len / 512) partitions
 *   partial_out [num_seqs][num_q_heads][P][head_dim] fp32   at offset 0
 *   partial_max [num_seqs][num_q_heads][P] fp32  (natural-log units)  next
 *   partial_sum [num_seqs][num_q_heads][P] fp32                         next
 * Offsets are given by pa_decode_split_workspace_offsets().
 */
size_t pa_decode_split_workspace_size(int num_seqs, int num_q_heads, int head_dim,
                                      int max_seq_len);
void pa_decode_split_workspace_offsets(int num_seqs, int num_q_heads, int head_dim,
                                       int max_seq_len, size_t *off_out, size_t *off_max,
                                       size_t *off_sum);

/*
 * pa_decode_split -- split-KV paged GQA decode.  Same result as pa_decode.
 * Pass 1: one CTA per (partition p, kv head, sequence) computes for its group
 * of query heads m_p = max of the scaled scores over tokens
 * [512 p, min(512 (p+1), L)), l_p = sum exp(s - m_p) and
 * o_p = sum exp(s - m_p) V / l_p, into the workspace (fp32).  Partitions at or
 * past ceil(L / 512) are neither written nor read; under a sliding window, neither
 * are those before the partition holding key L - sliding_window, whose tokens
 * before the window are left out of its m_p, l_p and o_p.
 * Pass 2 (merge): M = max_p m_p, w_p = l_p exp(m_p - M),
 * out = sum_p w_p o_p / sum_p w_p, rounded to bf16; L == 0 gives zeros.
 * max_seq_len must be >= every seq_lens[b]; a larger seq_len is clamped to it
 * and flagged PA_ERR_DEVICE_BOUNDS.  workspace is caller-owned device memory
 * of at least pa_decode_split_workspace_size() bytes, 256-byte aligned.
 */
int pa_decode_split(void *out, const void *q, const void *k_cache, const void *v_cache,
                    const int32_t *block_tables, const int32_t *seq_lens, int num_seqs,
                    int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                    int max_blocks_per_seq, int64_t num_blocks, int64_t stride_block,
                    int64_t stride_head, int64_t stride_token, float sm_scale,
                    int sliding_window, int kv_dtype, float k_scale, float v_scale,
                    int max_seq_len, void *workspace, size_t workspace_bytes, void *stream);

/*
 * The two passes of pa_decode_split as separate calls (same arguments and
 * workspace): pa_decode_partitions writes the per-partition (m_p, l_p, o_p)
 * into the workspace; pa_decode_merge reads them and writes out.  Both passes
 * must be given the same sliding_window.
 * pa_decode_split == pa_decode_partitions followed by pa_decode_merge.
 */
int pa_decode_partitions(const void *q, const void *k_cache, const void *v_cache,
                         const int32_t *block_tables, const int32_t *seq_lens, int num_seqs,
                         int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                         int max_blocks_per_seq, int64_t num_blocks, int64_t stride_block,
                         int64_t stride_head, int64_t stride_token, float sm_scale,
                         int sliding_window, int kv_dtype, float k_scale, float v_scale,
                         int max_seq_len, void *workspace, size_t workspace_bytes,
                         void *stream);
int pa_decode_merge(void *out, const int32_t *seq_lens, int num_seqs, int num_q_heads,
                    int head_dim, int max_seq_len, int sliding_window, const void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * pa_decode_split_static -- pa_decode_split for callers that cannot allocate.
 * (Not an operation from the reference pages: it has no counterpart there.)
 * Some callers may not call cudaMalloc and have no workspace to pass: e.g. a
 * plugin inside an engine that owns all device memory, or a latency-critical
 * decode loop where an allocation could synchronise the device or fail with
 * out-of-memory mid-step.  This entry point allocates nothing: the split
 * partials live in a device array of PA_STATIC_SCRATCH_BYTES compiled into the
 * library (every GPU that loads the library holds it until the process exits).
 * Arguments and result are those of pa_decode_split without the workspace.
 *  - The first call on a device (with that device current) looks up the
 *    array's device address with cudaGetSymbolAddress; make that first call
 *    before any stream capture.  The address is cached per device together
 *    with the id of the CUDA context it was looked up in; after a
 *    cudaDeviceReset the next call looks it up again (so, after a reset, that
 *    call too must come before any capture).
 *  - A batch whose pa_decode_split_workspace_size() exceeds
 *    PA_STATIC_SCRATCH_BYTES is rejected with PA_ERR_WORKSPACE.  The 16 MiB
 *    fit a 64-sequence, 32-head, head_dim-128 batch with seq_lens up to 4096
 *    (about 8.1 MiB of partials); 8 such sequences of up to 131072 tokens need
 *    about 32.5 MiB and must use pa_decode_split with a workspace.
 *  - All calls on a device share the array, which keeps the last call's
 *    partials; nothing in it needs clearing (each call writes every partition
 *    it later merges).  Calls that overlap on the GPU (e.g. on two streams of
 *    one device) race on the array: order them on one stream or with events.
 */
#define PA_STATIC_SCRATCH_BYTES (16 * 1024 * 1024)
int pa_decode_split_static(void *out, const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *block_tables, const int32_t *seq_lens, int num_seqs,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           int max_blocks_per_seq, int64_t num_blocks, int64_t stride_block,
                           int64_t stride_head, int64_t stride_token, float sm_scale,
                           int sliding_window, int kv_dtype, float k_scale, float v_scale,
                           int max_seq_len, void *stream);

/*
 * Bytes of workspace pa_ragged_prefill needs: 256 bytes of work counters, then room
 * for a device-built tile schedule.
 */
size_t pa_ragged_prefill_workspace_size(int batch, int total_qo_rows, int num_q_heads,
                                        int head_dim);

/*
 * pa_ragged_prefill -- ragged causal (or full) prefill, N requests, one launch.
 * Request r owns query rows [qo_indptr[r], qo_indptr[r+1]) and
 * kv_len_r = kv_indptr[r+1] - kv_indptr[r] keys.  Query row i of request r,
 * head h, attends to keys j < kv_len_r of kv head h / (num_q_heads/num_kv_heads)
 * and, if causal != 0, only to j <= i + (kv_len_r - qo_len_r) (bottom-right
 * alignment: the query rows are the LAST qo_len_r positions).  Under a sliding
 * window, row i sees only keys j > i + (kv_len_r - qo_len_r) - sliding_window.
 * A row with no visible key is written as zeros.
 *   o, q  [total_qo_rows][num_q_heads][head_dim] bf16
 *   Contiguous mode (block_tables == NULL): k, v are
 *         [total_kv_rows][num_kv_heads][head_dim] bf16 and key j of request r
 *         is row kv_indptr[r] + j; the stride arguments are ignored.
 *   Paged mode (block_tables != NULL): k, v are the paged pools, key j of
 *         request r is token j of block_tables[r] (as in pa_decode); the
 *         kv_indptr values only give the lengths.
 *   qo_indptr_h, kv_indptr_h  [batch+1] int32 HOST copies (used to size and
 *         order the launch: up to 1024 query tiles, the heaviest-first work list
 *         is built from them on the host and passed with the launch); qo_indptr_d,
 *         kv_indptr_d the same on the device, which must hold the same values.
 *   workspace  >= pa_ragged_prefill_workspace_size() bytes, 256-byte aligned, owned
 *         by the caller and used by one call at a time.  Its first 8 bytes are the
 *         launch's work counters: they must be zero before the first call (allocate
 *         it zeroed), and every call leaves them zero.  After a call that reported
 *         PA_ERR_TIMEOUT through pa_get_device_status, zero them again.
 *   sm_scale must be positive and finite (PA_ERR_INVALID otherwise).
 */
int pa_ragged_prefill(void *o, const void *q, const void *k, const void *v,
                      const int32_t *qo_indptr_h, const int32_t *kv_indptr_h,
                      const int32_t *qo_indptr_d, const int32_t *kv_indptr_d,
                      const int32_t *block_tables, int max_blocks_per_seq, int block_size,
                      int64_t num_blocks, int64_t stride_block, int64_t stride_head,
                      int64_t stride_token, int batch, int total_qo_rows,
                      int total_kv_rows, int num_q_heads, int num_kv_heads, int head_dim,
                      float sm_scale, int causal, int sliding_window, void *workspace,
                      size_t workspace_bytes, void *stream);

/*
 * Verification of drafted tokens.  Each sequence b of a step carries a tree of
 * T_b = qo_indptr[b+1] - qo_indptr[b] drafted nodes whose K/V rows are already in
 * its cache (pa_write_cache) as its LAST T_b tokens: seq_lens[b] counts them, the
 * context is the first C_b = seq_lens[b] - T_b tokens, node i is token C_b + i.
 */

/* Bytes of workspace pa_tree_decode needs (256-byte aligned; nothing in it has to be
 * initialised, and no call leaves anything in it for the next). */
size_t pa_tree_decode_workspace_size(int num_seqs, int max_tree_len, int num_q_heads,
                                     int num_kv_heads, int head_dim);

/*
 * pa_tree_decode -- attention of every drafted node, all sequences in one call.
 * Row qo_indptr[b] + i (node i of sequence b), head h, attends to
 *   - the context tokens j < C_b (under a sliding window those with
 *     j >= C_b + n_i - sliding_window, n_i the number of nodes its mask names), and
 *   - the nodes j < T_b whose bit is set in its mask row: bit j % 64 of word
 *     tree_mask[row][j / 64].  A node sees itself only if its own bit is set; any
 *     mask is allowed, not only those of trees, and bits at or past T_b are ignored.
 *     The window hides no node: for a path longer than it, clear the bits of the ancestors
 *     that have left it (n_i is then sliding_window, and no context token is seen).
 * A row that sees nothing is written as zeros.  Nodes it does not see and tokens past
 * seq_lens[b] contribute nothing, whatever their K/V rows hold (NaN included).
 *   out, q        [total_rows][num_q_heads][head_dim] bf16; rows outside
 *                 [qo_indptr[0], qo_indptr[num_seqs]) are neither read nor written
 *   qo_indptr     [num_seqs + 1] int32, device
 *   tree_mask     [total_rows][mask_words] 64-bit words, device, 8-byte aligned;
 *                 mask_words >= ceil(max_tree_len / 64)
 *   max_tree_len  >= every T_b, at most PA_MAX_TREE_LEN
 * A sequence whose T_b is negative, exceeds max_tree_len or seq_lens[b], whose rows leave
 * [0, total_rows), or whose seq_lens[b] exceeds max_blocks_per_seq * block_size (its nodes
 * are not in the table) is skipped (its rows are not written) and sets
 * PA_ERR_DEVICE_BOUNDS.  Block tables, pools, kv_dtype and scales are those of
 * pa_decode; sm_scale must be positive and finite.  The call reads qo_indptr, lengths
 * and masks on the device only, so a captured call can be replayed with new trees.
 */
#define PA_MAX_TREE_LEN 256
int pa_tree_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
                   const int32_t *block_tables, const int32_t *seq_lens,
                   const int32_t *qo_indptr, const int64_t *tree_mask, int mask_words,
                   int num_seqs, int total_rows, int max_tree_len, int num_q_heads,
                   int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                   int64_t num_blocks, int64_t stride_block, int64_t stride_head,
                   int64_t stride_token, float sm_scale, int sliding_window, int kv_dtype,
                   float k_scale, float v_scale, void *workspace, size_t workspace_bytes,
                   void *stream);

/*
 * pa_tree_commit -- after verification: the K/V rows of the accepted nodes become the
 * tokens right behind the context, in every one of the pools (all layers' K and V).
 * For sequence b and i < accept_lens[b], token C_b + i of each pool becomes what token
 * C_b + accepted[b][i] was, bit for bit, and new_seq_lens[b] = C_b + accept_lens[b].
 *   pools         HOST array of num_pools device pointers, all with the same strides,
 *                 kv_dtype and block tables (e.g. [k_0, v_0, k_1, v_1, ...]); a pool that
 *                 layers share is listed once
 *   accepted      [num_seqs][max_accept] int32 node indices, each greater than the one
 *                 before it (a path from the root down); entries past accept_lens[b]
 *                 are not read
 *   accept_lens   [num_seqs] int32
 *   new_seq_lens  [num_seqs] int32, written; shares no memory with what the call reads
 * A path is cut before its first entry that is out of range or not ascending, and
 * before max_accept entries; a sequence whose T_b is negative or exceeds max_tree_len
 * or seq_lens[b], or whose seq_lens[b] exceeds max_blocks_per_seq * block_size, keeps its
 * length and rows; both set PA_ERR_DEVICE_BOUNDS.  A page id outside the pool is neither
 * read nor written and sets it too.  Pages that hold
 * drafted tokens must belong to one sequence only.  One launch per 128 pools.
 */
int pa_tree_commit(void *const *pools, int num_pools, const int32_t *block_tables,
                   const int32_t *seq_lens, const int32_t *qo_indptr, const int32_t *accepted,
                   const int32_t *accept_lens, int32_t *new_seq_lens, int num_seqs,
                   int max_tree_len, int max_accept, int num_kv_heads, int head_dim,
                   int block_size, int max_blocks_per_seq, int64_t num_blocks,
                   int64_t stride_block, int64_t stride_head, int64_t stride_token,
                   int kv_dtype, void *stream);

/*
 * Decode over selected pages.  A long sequence's decode step reads only max_pages of
 * its pages per kv head: the first and the newest ones, and those whose keys can match
 * the step's query best by a bound kept per page.
 *
 * pa_page_bounds -- per page, kv head and channel the smallest and the largest key
 * value: bounds[page][kh][0][d] = min, [1][d] = max over the rows of the page that lie
 * inside the sequence (a NaN among them gives NaN).  Rewrites, for each sequence, the
 * pages that hold a token >= first_tokens[b] (NULL: every page), so a step calls it
 * with the lengths before its pa_write_cache.
 *   bounds          [num_blocks][num_kv_heads][2][head_dim] of the pool's type (FP8
 *                   pools: E4M3 codes, without k_scale)
 *   max_new_tokens  >= seq_lens[b] - first_tokens[b] for every b (>= seq_lens[b] when
 *                   first_tokens is NULL); bounds the launch: pages beyond those that so
 *                   many tokens can touch are not rewritten and set PA_ERR_DEVICE_BOUNDS (0:
 *                   the call does nothing).  Pages x num_kv_heads of a sequence that pass
 *                   2^31 are refused with PA_ERR_UNSUPPORTED.
 * A page that two sequences share must have the same rows in both.
 */
int pa_page_bounds(void *bounds, const void *k_cache, const int32_t *block_tables,
                   const int32_t *seq_lens, const int32_t *first_tokens, int max_new_tokens,
                   int num_seqs, int num_kv_heads, int head_dim, int block_size,
                   int max_blocks_per_seq, int64_t num_blocks, int64_t stride_block,
                   int64_t stride_head, int64_t stride_token, int kv_dtype, void *stream);

/* Bytes of workspace pa_select_pages needs (256-byte aligned, never initialised). */
size_t pa_select_pages_workspace_size(int num_seqs, int num_kv_heads, int max_blocks_per_seq);

/*
 * pa_select_pages -- the pages each (sequence, kv head) reads this step.  With n =
 * ceil(seq_lens[b] / block_size) pages, min(n, max_pages) are chosen: the first
 * sink_pages, the last recent_pages, and of the others those of the largest score
 *   score(p) = sum over the kv head's query heads h and the channels d of
 *              max(q[b][h][d] * min_p[d], q[b][h][d] * max_p[d]),
 * an upper bound of the sum of q . k over any key of the page (where a head's q is zero the
 * channel adds nothing, an infinite bound included).  Scores are compared as
 * exact numbers (candidates that 32 bits cannot tell apart are scored again in 64);
 * equal scores go to the lower page, and a NaN score counts as the largest.
 *   page_tables  [num_seqs][num_kv_heads][max_pages] int32, written whole: the chosen
 *                pages' ids in the order of their tokens, then -1
 *   page_lens    [num_seqs] int32, written: the number of tokens those pages hold
 * max_pages > 0, sink_pages >= 0, recent_pages >= 1 (a newest page's bounds may lag its
 * rows), sink_pages + recent_pages <= max_pages, max_blocks_per_seq <= 524288.  A page id
 * outside the pool scores lowest and sets PA_ERR_DEVICE_BOUNDS.  page_tables and page_lens
 * share no memory with block_tables, seq_lens or one another.
 */
int pa_select_pages(int32_t *page_tables, int32_t *page_lens, const void *q, const void *bounds,
                    const int32_t *block_tables, const int32_t *seq_lens, int num_seqs,
                    int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                    int max_blocks_per_seq, int64_t num_blocks, int max_pages, int sink_pages,
                    int recent_pages, int kv_dtype, void *workspace, size_t workspace_bytes,
                    void *stream);

/*
 * pa_decode_pages -- the split decode with one page list per (sequence, kv head): the
 * query heads of kv head kh attend over the page_lens[b] tokens of the pages
 * page_tables[b][kh], as pa_decode_split over a block table does.  Wide groups at head_dim 64
 * and 256 run on the tree kernel, whose roundings differ from that call's, where num_seqs,
 * num_kv_heads and max_pages multiply to enough reading.  Takes what pa_select_pages writes,
 * or any lists whose pages are full but the last; an empty one gives zeros.
 * workspace: pa_decode_split_workspace_size(num_seqs, num_q_heads, head_dim,
 * max_pages * block_size) bytes, 256-byte aligned.
 */
int pa_decode_pages(void *out, const void *q, const void *k_cache, const void *v_cache,
                    const int32_t *page_tables, const int32_t *page_lens, int num_seqs,
                    int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                    int max_pages, int64_t num_blocks, int64_t stride_block,
                    int64_t stride_head, int64_t stride_token, float sm_scale, int kv_dtype,
                    float k_scale, float v_scale, void *workspace, size_t workspace_bytes,
                    void *stream);

/*
 * Rotary positions.  The token at position P turns its channels pair by pair: pair i of
 * R / 2 (R = rotary_dim) by the angle a = P * f_i,
 *   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a),
 * where (x1, x2) are channels (i, i + R / 2), or (2 i, 2 i + 1) if interleaved != 0, and m
 * is the attention factor.  Channels from R on pass unchanged.  The angle is held to 2^-24
 * of a half turn at positions up to 2^31, products and sums are fp32, each result is
 * rounded once.
 *
 * Frequencies come as a table of rotary_dim / 2 numbers made once per model on the HOST
 * and copied to the device: entry i is the fraction of a turn per position, in units of
 * 2^-64, the nearest one (of bases beyond 2^900, to the 53 bits of a double).
 *
 * pa_rope_table writes the table and the attention factor of f_i = base^(-2 i / R) under a
 * scaling for long contexts by factor s:
 *   PA_ROPE_NONE    f_i
 *   PA_ROPE_LINEAR  f_i / s (positions interpolated)
 *   PA_ROPE_NTK     base * s^(R / (R - 2)) in place of base
 *   PA_ROPE_BANDS   by the turns t = original_len * f_i / 2 pi a pair makes in the original
 *                   context: f_i / s below `low` turns, f_i above `high`, between them
 *                   f_i ((1 - r) / s + r) with r = (t - low) / (high - low) (usual: 1, 4)
 *   PA_ROPE_YARN    f_i (r / s + 1 - r), r rising from 0 to 1 between the pair numbers
 *                   floor(n(high)) and ceil(n(low)), where n(t) = R ln(original_len /
 *                   (2 pi t)) / (2 ln base), cut to [0, R - 1] (usual: low 1, high 32);
 *                   attention factor 0.1 ln s + 1 for s > 1
 * (attention factor 1 for the others).  factor, low, high and original_len are read by the
 * scalings that name them.  pa_rope_table_of takes any other frequencies, in radians per
 * position.
 *   turns_h  [rotary_dim / 2] HOST; attention_factor_h HOST, may be NULL
 */
typedef enum {
    PA_ROPE_NONE = 0,
    PA_ROPE_LINEAR = 1,
    PA_ROPE_NTK = 2,
    PA_ROPE_BANDS = 3,
    PA_ROPE_YARN = 4
} pa_rope_scaling;
int pa_rope_table(uint64_t *turns_h, float *attention_factor_h, int rotary_dim, double base,
                  int scaling, double factor, double low, double high, int64_t original_len);
int pa_rope_table_of(uint64_t *turns_h, const double *frequencies_h, int num_pairs);

/*
 * pa_rope -- q and k of num_tokens tokens, turned to their positions.
 *   q, k          [num_tokens][heads][head_dim] bf16 by element strides (token, head), each
 *                 a multiple of 16 bytes; head_dim contiguous.  0 heads: not touched.
 *   q_out, k_out  the same shape by strides of their own; q_out may be q and k_out k with
 *                 the same strides (in place), else outputs share no memory with inputs or
 *                 one another.  Slices of one buffer are seen to be apart where they lie
 *                 beside one another in the stride of their tokens (or heads, if larger), or
 *                 their rows do in a common divisor of all strides ([heads][3][head_dim]);
 *                 other interleavings are refused
 *   positions     [num_tokens] int64, any value (negative ones turn back)
 *   turns         [rotary_dim / 2], device, from pa_rope_table
 *   inverse       != 0: by -a.  That is the gradient of the call with inverse == 0 (the
 *                 transposed map), and takes its rotation back where m is 1.
 * head_dim in {64, 128, 256}, rotary_dim even, at most head_dim.
 */
int pa_rope(void *q_out, void *k_out, const void *q, const void *k, const int64_t *positions,
            const uint64_t *turns, int64_t num_tokens, int num_q_heads, int num_k_heads,
            int head_dim, int rotary_dim, int64_t q_out_stride_token, int64_t q_out_stride_head,
            int64_t k_out_stride_token, int64_t k_out_stride_head, int64_t q_stride_token,
            int64_t q_stride_head, int64_t k_stride_token, int64_t k_stride_head,
            int interleaved, int inverse, float attention_factor, void *stream);

/*
 * pa_rope_append -- pa_rope and pa_write_cache in one pass: q turned into q_out, k turned
 * into the cache at slot_mapping, v into the cache as it is.  An FP8 pool takes the E4M3
 * codes of the turned fp32 values (k_scale, v_scale as in pa_write_cache).
 *   q, k, v, q_out  as in pa_rope (num_q_heads may be 0; k, v share num_kv_heads); none of
 *                   them lies in the caches
 *   slot_mapping    [num_tokens] int64; a token whose slot is negative is padding: nothing of
 *                   it is written, its row of q_out included.  A slot outside the pool is
 *                   treated the same and sets PA_ERR_DEVICE_BOUNDS.  Of two tokens with the
 *                   same slot in one call, each channel there is one's or the other's
 */
int pa_rope_append(void *q_out, const void *q, const void *k, const void *v, void *k_cache,
                   void *v_cache, const int64_t *slot_mapping, const int64_t *positions,
                   const uint64_t *turns, int64_t num_tokens, int num_q_heads,
                   int num_kv_heads, int head_dim, int rotary_dim, int block_size,
                   int64_t num_blocks, int64_t q_out_stride_token, int64_t q_out_stride_head,
                   int64_t q_stride_token, int64_t q_stride_head, int64_t k_stride_token,
                   int64_t k_stride_head, int64_t v_stride_token, int64_t v_stride_head,
                   int64_t stride_block, int64_t stride_head, int64_t stride_token,
                   int interleaved, float attention_factor, int kv_dtype, float k_scale,
                   float v_scale, void *stream);

/*
 * Beam search.  A request has num_beams beams, each a sequence of its own in the cache:
 * sequence r * num_beams + b.  A step runs the model on every beam's newest token, chooses
 * the best continuations (pa_beam_select) and lets the cache follow them
 * (pa_beam_reorder with parents = the chosen beams).
 */
#define PA_MAX_BEAMS 32          /* num_beams */
#define PA_MAX_BEAM_OUT 64       /* num_out */
#define PA_MAX_BEAM_VOCAB (1 << 24)
typedef enum { PA_LOGITS_F32 = 0, PA_LOGITS_BF16 = 1 } pa_logits_dtype;

/* Bytes of workspace pa_beam_select needs (256-byte aligned; nothing in it has to be
 * initialised, and no call leaves anything in it for the next). */
size_t pa_beam_select_workspace_size(int num_requests, int num_beams, int vocab);

/*
 * pa_beam_select -- for every request the num_out best of all pairs (beam b, token t) by
 *   score = cum_scores[r][b] + x_t - log sum_u exp x_u,   x the beam's row of logits,
 * best first; equal scores go to the lower beam, then to the lower token.  Scores are
 * compared as sums of two fp32; a row's log-sum-exp is known to 2^-17, so pairs of two beams whose
 * scores are closer than 2^-16 may come in either order.  Equal rows have equal sums.
 *   logits      [num_requests * num_beams] rows of vocab values of logits_dtype, stride_row
 *               elements apart (rows of any alignment; multiples of 16 bytes are faster).
 *               -inf rules a token out.
 *   cum_scores  [num_requests][num_beams] fp32.  -inf takes a beam out, whatever its logits
 *               hold (a first step has one beam at 0 and the others at -inf).
 *   finished    [num_requests][num_beams] bytes, or NULL.  A beam with a nonzero flag offers
 *               one pair, end_token at the score cum_scores, whatever its logits hold.
 *   scores      [num_requests][num_out] fp32, beams and tokens [num_requests][num_out] int32,
 *               written whole: behind the pairs there are, -inf, -1 and -1.  A pair whose
 *               score rounds to -inf is none.
 * A beam whose logits hold NaN or +inf, or whose cum_scores is one of them, offers nothing
 * and sets the PA_ERR_INVALID bit of the device status word.  The outputs share no memory
 * with what the call reads or one another.  Two launches; one where there are few requests
 * and the stream is not being captured, with the same result.
 */
int pa_beam_select(float *scores, int32_t *beams, int32_t *tokens, const void *logits,
                   const float *cum_scores, const uint8_t *finished, int end_token,
                   int num_requests, int num_beams, int vocab, int num_out,
                   int64_t stride_row, int logits_dtype, void *workspace,
                   size_t workspace_bytes, void *stream);

/*
 * pa_beam_reorder -- the cache follows the chosen beams: sequence j of each request goes on
 * from what sequence p = parents[r][j] held, in every one of the pools.  With L its length,
 *   - its block-table row takes p's ids of the full pages (the first L / block_size): full
 *     pages are shared, not copied;
 *   - the L % block_size rows of the page that its next token goes to become p's rows, bit
 *     for bit.  That page, block_tables[j][L / block_size], must be named by no other
 *     sequence; the entry stays.
 * All sequences move at once: p's rows and ids are those before the call.  A sequence that
 * is its own parent stays as it is.  So does one with parents -1, which is out of the
 * search: its page may be another's by now.  After a prompt whose pages the beams share,
 * parents 0 and a page of its own at L / block_size make each beam's copy of the last one.
 *   pools         HOST array of num_pools device pointers, as in pa_tree_commit
 *   block_tables  [num_requests * num_beams][max_blocks_per_seq], changed in place
 *   seq_lens      [num_requests * num_beams]; parents [num_requests][num_beams] int32
 * A sequence is left as it is and PA_ERR_DEVICE_BOUNDS set where its parent is no beam of
 * the request or has another length, the length is negative or passes the table, or (unless L %
 * block_size is 0) its own or its parent's page is not in the pool or its own is that of
 * another beam in the search.  Pages that no sequence names any more are the caller's to find.
 * Where pa_block_table_sync keeps the table, the rows of its host copy are to be moved
 * likewise, or the next upload of one brings back what it was.  One launch per 128 pools.
 */
int pa_beam_reorder(void *const *pools, int num_pools, int32_t *block_tables,
                    const int32_t *seq_lens, const int32_t *parents, int num_requests,
                    int num_beams, int num_kv_heads, int head_dim, int block_size,
                    int max_blocks_per_seq, int64_t num_blocks, int64_t stride_block,
                    int64_t stride_head, int64_t stride_token, int kv_dtype, void *stream);

/*
 * Block-table upload for CUDA-graph replays ("libmir-cuda attention/mod.rs",
 * the captured decode nodes and their block-table snapshot; "paged_attn.py",
 * block tables padded for graph capture): a captured decode reads a fixed
 * device table, so between replays only the rows that changed need copying.
 *   host_table   [num_rows][row_len] int32, the table the caller wants on the
 *                device (any host memory);
 *   snapshot     [num_rows][row_len] int32 PINNED host memory owned by the
 *                caller, holding what was last uploaded.  Before the first
 *                call, fill it with -1 (a value no row holds), so that the
 *                first call finds every row changed and uploads the whole
 *                table;
 *   device_table [num_rows][row_len] int32 device memory.
 * Rows of host_table that differ from the snapshot are copied into it, and
 * each run of consecutive changed rows is enqueued on `stream` as one async
 * copy from the snapshot to device_table.  *rows_uploaded (if not NULL)
 * receives the number of rows copied.  The snapshot's rows must not change
 * again until the stream has executed those copies (for instance, sync once
 * per step, after the previous step's work on the stream is done).
 * Returns PA_OK, PA_ERR_INVALID or PA_ERR_CUDA.
 */
int pa_block_table_sync(const int32_t *host_table, int32_t *snapshot, int32_t *device_table,
                        int num_rows, int row_len, int *rows_uploaded, void *stream);

/*
 * Whole-page copies ("paged_attn.py", PagedAttention.copy_blocks and
 * PagedAttention.swap_blocks).  A page of a pool is the block_bytes contiguous
 * bytes at byte offset page * block_bytes (block_bytes = stride_block * element
 * size for a dense pool of either page layout); block_bytes must be a positive
 * multiple of 16 and every pool 16-byte aligned.
 * block_mapping is [num_pairs][2] int64 (source page, destination page).  For
 * each pair and each pool, the source page's bytes become the destination
 * page's bytes, bit for bit.  A pair with a negative entry is skipped (padding);
 * a pair with a source >= the source pool's block count or a destination >=
 * the destination pool's block count is skipped and sets PA_ERR_DEVICE_BOUNDS
 * in the device status word.  A destination that appears twice, or that is
 * also a source in the same call, gives an unspecified result.  One kernel
 * launch moves every (pair, pool) of a call (one launch per 128 pools); the
 * calls allocate nothing and return once the work is enqueued on `stream`.
 */

/*
 * pa_copy_blocks -- copy_blocks: the pairs are applied inside each of the
 * num_pools pools (pass every layer's key pool and value pool, e.g.
 * [k_0, v_0, k_1, v_1, ...]); all pools have num_blocks pages.
 *   pools          HOST array of num_pools device pointers
 *   block_mapping  device memory (or pinned host memory whose device address
 *                  equals its host address, as cudaHostAlloc gives), read by
 *                  the kernel; the call makes no CUDA runtime query, so it can
 *                  be captured into a CUDA graph.
 * Returns PA_OK, PA_ERR_INVALID or PA_ERR_CUDA.
 */
int pa_copy_blocks(void *const *pools, int num_pools, const int64_t *block_mapping,
                   int64_t num_pairs, int64_t num_blocks, int64_t block_bytes, void *stream);

/*
 * pa_swap_blocks -- swap_blocks: pool i of src_pools (src_num_blocks pages)
 * into pool i of dst_pools (dst_num_blocks pages), for i < num_pools <= 4096.
 * Each pool and block_mapping may be device memory of the current device or
 * pinned host memory (cudaHostAlloc / cudaHostRegister), or any host memory on
 * a device that can read pageable memory; host pages are read and written by
 * the kernel directly over the CPU-GPU link.  The host addresses are resolved
 * with cudaPointerGetAttributes on every call (capture this call only where that
 * query is allowed).  Memory that the device cannot address is rejected with
 * PA_ERR_INVALID.  Host memory must stay valid and unchanged until the stream
 * has run the copy.
 *   src_pools, dst_pools  HOST arrays of num_pools pointers
 * Returns PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED or PA_ERR_CUDA.
 */
int pa_swap_blocks(const void *const *src_pools, void *const *dst_pools, int num_pools,
                   const int64_t *block_mapping, int64_t num_pairs, int64_t src_num_blocks,
                   int64_t dst_num_blocks, int64_t block_bytes, void *stream);

/*
 * Synchronises `stream`, then reads and clears the current device's status
 * word: *status_h receives PA_OK or the OR-ed PA_ERR_* bits recorded by the
 * device-side guards (bit (1 << code)).  Returns PA_OK or PA_ERR_CUDA.
 */
int pa_get_device_status(int *status_h, void *stream);

/*
 * pa_selftest_wait_timeout -- exercises the bounded wait that every kernel's
 * pipeline uses.  One thread waits on an mbarrier that nothing completes; after
 * about 1 s (the per-wait limit) it records PA_ERR_TIMEOUT in the device status
 * word and the kernel returns.  No memory is touched but that word; the context
 * stays usable.  Enqueued on `stream`; returns PA_OK, or PA_ERR_CUDA when the
 * launch fails.
 */
int pa_selftest_wait_timeout(void *stream);

/* Thread-local description of the last error returned on this thread. */
const char *pa_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* PA_H */
