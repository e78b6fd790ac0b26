"""Paged-KV GQA attention for GB300 (sm_103a).

A thin ctypes binding over the C ABI in include/pa.h (libpa.so, built in-tree
by ``paged_kv_gqa_15_gb300.build``).  Functions take torch CUDA tensors and
only marshal pointers, shapes and strides: every step of the computation runs
in the library's CUDA kernels.  There is no CPU fallback -- if libpa.so is
missing or fails to load, every call raises.
"""
from __future__ import annotations

import array
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")
PARTITION_TOKENS = 512
PAGE_TOKENS = 16
_lib = None

PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_CUDA, PA_ERR_WORKSPACE, PA_ERR_TIMEOUT, \
    PA_ERR_DEVICE_BOUNDS = range(7)
PA_KV_BF16, PA_KV_FP8_E4M3 = 0, 1   # pa_kv_dtype
STATUS_NAMES = {1: "INVALID", 2: "UNSUPPORTED", 3: "CUDA", 4: "WORKSPACE", 5: "TIMEOUT",
                6: "DEVICE_BOUNDS"}


class PaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"pa error {code} ({STATUS_NAMES.get(code, '?')}): {msg}")
        self.code = code


def load():
    """Load libpa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library {LIB_PATH} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, L, F, Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                     ctypes.c_size_t)
    lib.pa_write_cache.argtypes = [P, P, P, P, P, L, I, I, I, L, L, L, L, I, F, F, P]
    lib.pa_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, L, L, L, L, F, I, I, F, F, P]
    lib.pa_decode_split_workspace_size.argtypes = [I, I, I, I]
    lib.pa_decode_split_workspace_size.restype = Z
    lib.pa_decode_split_workspace_offsets.argtypes = [I, I, I, I, P, P, P]
    lib.pa_decode_split_workspace_offsets.restype = None
    lib.pa_decode_split.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, L, L, L, L, F, I, I, F,
                                    F, I, P, Z, P]
    lib.pa_decode_partitions.argtypes = [P, P, P, P, P, I, I, I, I, I, I, L, L, L, L, F, I, I, F,
                                         F, I, P, Z, P]
    lib.pa_decode_merge.argtypes = [P, P, I, I, I, I, I, P, Z, P]
    lib.pa_decode_split_static.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, L, L, L, L, F, I,
                                           I, F, F, I, P]
    lib.pa_decode_split_static.restype = I
    lib.pa_ragged_prefill_workspace_size.argtypes = [I, I, I, I]
    lib.pa_ragged_prefill_workspace_size.restype = Z
    lib.pa_ragged_prefill.argtypes = [P, P, P, P, P, P, P, P, P, I, I, L, L, L, L, I, I, I, I, I,
                                      I, F, I, I, P, Z, P]
    lib.pa_get_device_status.argtypes = [P, P]
    lib.pa_selftest_wait_timeout.argtypes = [P]
    lib.pa_block_table_sync.argtypes = [P, P, P, I, I, P, P]
    lib.pa_block_table_sync.restype = I
    lib.pa_copy_blocks.argtypes = [P, I, P, L, L, L, P]
    lib.pa_copy_blocks.restype = I
    lib.pa_swap_blocks.argtypes = [P, P, I, P, L, L, L, L, P]
    lib.pa_swap_blocks.restype = I
    lib.pa_decode_pages.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, L, L, L, L, F, I, F, F, P,
                                    Z, P]
    lib.pa_tree_decode_workspace_size.argtypes = [I, I, I, I, I]
    lib.pa_tree_decode_workspace_size.restype = Z
    lib.pa_tree_decode.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, L, L, L, L, F,
                                   I, I, F, F, P, Z, P]
    lib.pa_tree_commit.argtypes = [P, I, P, P, P, P, P, P, I, I, I, I, I, I, I, L, L, L, L, I, P]
    lib.pa_page_bounds.argtypes = [P, P, P, P, P, I, I, I, I, I, I, L, L, L, L, I, P]
    lib.pa_select_pages_workspace_size.argtypes = [I, I, I]
    lib.pa_select_pages_workspace_size.restype = Z
    lib.pa_select_pages.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, L, I, I, I, I, P, Z, P]
    D = ctypes.c_double
    lib.pa_rope_table.argtypes = [P, P, I, D, I, D, D, D, L]
    lib.pa_rope_table_of.argtypes = [P, P, I]
    lib.pa_rope.argtypes = [P, P, P, P, P, P, L, I, I, I, I, L, L, L, L, L, L, L, L, I, I, F, P]
    lib.pa_rope_append.argtypes = [P, P, P, P, P, P, P, P, P, L, I, I, I, I, I, L, L, L, L, L, L, L, L,
                                   L, L, L, L, I, F, I, F, F, P]
    lib.pa_beam_select_workspace_size.argtypes = [I, I, I]
    lib.pa_beam_select_workspace_size.restype = Z
    lib.pa_beam_select.argtypes = [P, P, P, P, P, P, I, I, I, I, I, L, I, P, Z, P]
    lib.pa_beam_reorder.argtypes = [P, I, P, P, P, I, I, I, I, I, I, L, L, L, L, I, P]
    lib.pa_last_error.restype = ctypes.c_char_p
    for name in ("pa_write_cache", "pa_decode", "pa_decode_split", "pa_decode_partitions",
                 "pa_decode_merge", "pa_ragged_prefill", "pa_decode_pages", "pa_tree_decode",
                 "pa_tree_commit", "pa_page_bounds", "pa_select_pages", "pa_rope_table",
                 "pa_rope_table_of", "pa_rope", "pa_rope_append", "pa_beam_select",
                 "pa_beam_reorder",
                 "pa_get_device_status"):
        getattr(lib, name).restype = I
    _lib = lib
    return lib


def _check(rc: int):
    if rc != PA_OK:
        raise PaError(rc, load().pa_last_error().decode())


def _ptr(t):
    # ctypes takes a plain address for a void *: no object per argument and call
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object (2.5 us of a call's host time), where torch
# has the call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None):
    """The stream's handle, or the current one's of the current device, if the caller knows that."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device() if device is None else device)
    return torch.cuda.current_stream().cuda_stream


def pool_strides(cache: torch.Tensor, layout: str = "HND"):
    """(block, head, token) element strides of a 4-D pool tensor.

    HND: [num_blocks][num_kv_heads][block_size][head_dim];
    NHD: [num_blocks][block_size][num_kv_heads][head_dim]."""
    s = cache.stride()
    assert len(s) == 4 and s[3] == 1, "pool must be 4-D with a contiguous head_dim"
    return (s[0], s[1], s[2]) if layout == "HND" else (s[0], s[2], s[1])


_FP8_DTYPES = (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))


def kv_dtype_of(cache: torch.Tensor) -> int:
    """pa_kv_dtype of a pool tensor: bf16, or FP8 E4M3 codes (float8_e4m3fn or uint8)."""
    dtype = cache.dtype
    if dtype == torch.bfloat16:
        return PA_KV_BF16
    if dtype in _FP8_DTYPES:
        return PA_KV_FP8_E4M3
    raise TypeError(f"unsupported KV cache dtype {dtype}")


def _pool_geometry(cache, layout):
    nb, a, b, hd = cache.shape
    return (nb, a, b, hd) if layout == "HND" else (nb, b, a, hd)


def _host_ptr(a):
    """Address of a C-contiguous host array (numpy or CPU torch tensor)."""
    if isinstance(a, torch.Tensor):
        assert a.device.type == "cpu" and a.is_contiguous()
        return ctypes.c_void_p(a.data_ptr())
    assert a.flags["C_CONTIGUOUS"]
    return ctypes.c_void_p(a.ctypes.data)


def pa_block_table_sync(host_table, snapshot, device_table, stream=None) -> int:
    """Uploads the rows of host_table (int32 [rows, cols], host) that differ from
    snapshot (a pinned int32 host tensor holding what was last uploaded) into
    device_table, refreshing the snapshot; returns the number of rows copied."""
    rows, cols = host_table.shape
    assert tuple(snapshot.shape) == (rows, cols) and tuple(device_table.shape) == (rows, cols)
    n = ctypes.c_int(0)
    _check(load().pa_block_table_sync(_host_ptr(host_table), _host_ptr(snapshot),
                                      _ptr(device_table), rows, cols, ctypes.byref(n),
                                      _stream(stream) if torch.cuda.is_available() else None))
    return n.value


def _page_geometry(pools):
    """(num_blocks, block_bytes) shared by a list of pools, each [num_blocks, ...] with
    densely packed pages (page b = bytes [b * block_bytes, (b + 1) * block_bytes))."""
    nb, bb = None, None
    for t in pools:
        page_elems = t[0].numel() if t.shape[0] > 0 else 0
        assert t.stride(0) == page_elems and t[0].is_contiguous(), \
            "pool pages must be densely packed"
        b = page_elems * t.element_size()
        assert (nb, bb) in ((None, None), (t.shape[0], b)), "pools differ in geometry"
        nb, bb = t.shape[0], b
    return nb, bb


def _pointer_array(tensors):
    return (ctypes.c_void_p * max(1, len(tensors)))(*[t.data_ptr() for t in tensors])


def pa_copy_blocks(key_caches, value_caches, block_mapping, stream=None):
    """copy_blocks: for every (src, dst) row of block_mapping (int64 [n, 2], on the
    device), page src of every layer's key and value pool is copied to page dst."""
    pools = [t for kv in zip(key_caches, value_caches) for t in kv]
    if not pools or block_mapping.numel() == 0:
        return
    assert block_mapping.dtype == torch.int64 and block_mapping.is_contiguous()
    nb, bb = _page_geometry(pools)
    _check(load().pa_copy_blocks(_pointer_array(pools), len(pools), _ptr(block_mapping),
                                 block_mapping.shape[0], nb, bb, _stream(stream)))


def pa_swap_blocks(src, dst, block_mapping, stream=None):
    """swap_blocks: page src of each source pool to page dst of the matching
    destination pool, for every row of block_mapping (int64 [n, 2]).  src / dst are a
    pool or a list of pools, each on the device or in pinned host memory; the mapping
    may be on either side too."""
    src = list(src) if isinstance(src, (list, tuple)) else [src]
    dst = list(dst) if isinstance(dst, (list, tuple)) else [dst]
    assert len(src) == len(dst)
    if not src or block_mapping.numel() == 0:
        return
    assert block_mapping.dtype == torch.int64 and block_mapping.is_contiguous()
    snb, sbb = _page_geometry(src)
    dnb, dbb = _page_geometry(dst)
    assert sbb == dbb, "source and destination pages differ in size"
    _check(load().pa_swap_blocks(_pointer_array(src), _pointer_array(dst), len(src),
                                 _ptr(block_mapping), block_mapping.shape[0], snb, dnb, sbb,
                                 _stream(stream)))


def pa_write_cache(k, v, k_cache, v_cache, slot_mapping, layout="HND", stream=None,
                   k_scale=1.0, v_scale=1.0):
    """reshape_and_cache: scatter k/v [T, nkv, hd] into the pools at slot_mapping [T];
    an FP8 pool (float8_e4m3fn or uint8) stores the E4M3 codes of x / k_scale (v_scale)."""
    nb, nkv, bs, hd = _pool_geometry(k_cache, layout)
    sb, sh, st = pool_strides(k_cache, layout)
    _check(load().pa_write_cache(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(slot_mapping), k.shape[0], nkv, hd, bs, nb, sb, sh, st,
                                 kv_dtype_of(k_cache), float(k_scale), float(v_scale),
                                 _stream(stream)))


def pa_decode(out, q, k_cache, v_cache, block_tables, seq_lens, sm_scale, layout="HND",
              stream=None, sliding_window=0, k_scale=1.0, v_scale=1.0):
    """Single-pass paged GQA decode into out [B, nq, hd]; sliding_window > 0 keeps the
    last sliding_window keys of each sequence."""
    nb, nkv, bs, hd = _pool_geometry(k_cache, layout)
    sb, sh, st = pool_strides(k_cache, layout)
    B, nq, _ = q.shape
    _check(load().pa_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                            _ptr(seq_lens), B, nq, nkv, hd, bs, block_tables.shape[1], nb, sb,
                            sh, st, float(sm_scale), int(sliding_window), kv_dtype_of(k_cache),
                            float(k_scale), float(v_scale), _stream(stream)))


def decode_split_workspace_size(num_seqs, num_q_heads, head_dim, max_seq_len) -> int:
    return int(load().pa_decode_split_workspace_size(num_seqs, num_q_heads, head_dim,
                                                     max_seq_len))


def decode_split_workspace_views(workspace, num_seqs, num_q_heads, head_dim, max_seq_len):
    """(partial_out, partial_max, partial_sum) float32 views of a split workspace."""
    oo, om, ol = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    load().pa_decode_split_workspace_offsets(num_seqs, num_q_heads, head_dim, max_seq_len,
                                             ctypes.byref(oo), ctypes.byref(om),
                                             ctypes.byref(ol))
    P = (max_seq_len + PARTITION_TOKENS - 1) // PARTITION_TOKENS
    n = num_seqs * num_q_heads * P
    ws = workspace.view(torch.uint8)
    po = ws[oo.value:oo.value + n * head_dim * 4].view(torch.float32).view(num_seqs, num_q_heads,
                                                                           P, head_dim)
    pm = ws[om.value:om.value + n * 4].view(torch.float32).view(num_seqs, num_q_heads, P)
    pl = ws[ol.value:ol.value + n * 4].view(torch.float32).view(num_seqs, num_q_heads, P)
    return po, pm, pl


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """A zeroed, 256-byte-aligned uint8 device buffer of at least nbytes (the prefill's
    work counters must start at zero)."""
    buf = torch.zeros(max(int(nbytes), 1) + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + max(int(nbytes), 1)]


def pa_decode_split(out, q, k_cache, v_cache, block_tables, seq_lens, sm_scale, max_seq_len,
                    workspace, layout="HND", stream=None, sliding_window=0, k_scale=1.0,
                    v_scale=1.0):
    """Split-KV paged GQA decode (512-token partitions + LSE merge) into out [B, nq, hd]."""
    nb, nkv, bs, hd = _pool_geometry(k_cache, layout)
    sb, sh, st = pool_strides(k_cache, layout)
    B, nq, _ = q.shape
    _check(load().pa_decode_split(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(block_tables), _ptr(seq_lens), B, nq, nkv, hd, bs,
                                  block_tables.shape[1], nb, sb, sh, st, float(sm_scale),
                                  int(sliding_window), kv_dtype_of(k_cache), float(k_scale),
                                  float(v_scale), int(max_seq_len), _ptr(workspace),
                                  workspace.numel(), _stream(stream)))


STATIC_SCRATCH_BYTES = 16 * 1024 * 1024  # PA_STATIC_SCRATCH_BYTES in include/pa.h


def pa_decode_split_static(out, q, k_cache, v_cache, block_tables, seq_lens, sm_scale,
                           max_seq_len, layout="HND", stream=None, sliding_window=0,
                           k_scale=1.0, v_scale=1.0):
    """pa_decode_split with the library's fixed device scratch instead of a workspace,
    for callers that cannot allocate device memory.  Batches needing more than
    STATIC_SCRATCH_BYTES of partials are rejected; concurrent calls on one device race."""
    nb, nkv, bs, hd = _pool_geometry(k_cache, layout)
    sb, sh, st = pool_strides(k_cache, layout)
    B, nq, _ = q.shape
    _check(load().pa_decode_split_static(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                         _ptr(block_tables), _ptr(seq_lens), B, nq, nkv, hd, bs,
                                         block_tables.shape[1], nb, sb, sh, st, float(sm_scale),
                                         int(sliding_window), kv_dtype_of(k_cache),
                                         float(k_scale), float(v_scale), int(max_seq_len),
                                         _stream(stream)))


def pa_decode_partitions(q, k_cache, v_cache, block_tables, seq_lens, sm_scale, max_seq_len,
                         workspace, layout="HND", stream=None, sliding_window=0, k_scale=1.0,
                         v_scale=1.0):
    """Split-KV pass 1: per-partition (m, l, o) into the workspace."""
    nb, nkv, bs, hd = _pool_geometry(k_cache, layout)
    sb, sh, st = pool_strides(k_cache, layout)
    B, nq, _ = q.shape
    _check(load().pa_decode_partitions(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                       _ptr(seq_lens), B, nq, nkv, hd, bs, block_tables.shape[1],
                                       nb, sb, sh, st, float(sm_scale), int(sliding_window),
                                       kv_dtype_of(k_cache), float(k_scale), float(v_scale),
                                       int(max_seq_len), _ptr(workspace), workspace.numel(),
                                       _stream(stream)))


def pa_decode_merge(out, seq_lens, max_seq_len, workspace, stream=None, sliding_window=0):
    """Split-KV pass 2: log-sum-exp merge of the workspace partitions into out (the
    same sliding_window as pass 1)."""
    B, nq, hd = out.shape
    _check(load().pa_decode_merge(_ptr(out), _ptr(seq_lens), B, nq, hd, int(max_seq_len),
                                  int(sliding_window), _ptr(workspace), workspace.numel(),
                                  _stream(stream)))


def ragged_prefill_workspace_size(batch, total_qo_rows, num_q_heads, head_dim) -> int:
    return int(load().pa_ragged_prefill_workspace_size(batch, total_qo_rows, num_q_heads,
                                                       head_dim))


def pa_ragged_prefill(o, q, k, v, qo_indptr_h, kv_indptr_h, qo_indptr_d, kv_indptr_d, sm_scale,
                      causal=True, block_tables=None, num_kv_heads=None, layout="HND",
                      workspace=None, stream=None, sliding_window=0):
    """Ragged prefill.  Contiguous mode: k, v [total_kv, nkv, hd].  Paged mode
    (block_tables given): k, v are pools and kv_indptr only carries lengths.
    qo_indptr_h / kv_indptr_h are int32 host tensors (or numpy arrays)."""
    import numpy as np
    qh = np.ascontiguousarray(np.asarray(qo_indptr_h, np.int32))
    kh = np.ascontiguousarray(np.asarray(kv_indptr_h, np.int32))
    batch = qh.size - 1
    total_qo, nq, hd = q.shape
    if block_tables is None:
        nkv = k.shape[1]
        nb, bs, sb, sh, st, mb = 1, 16, 8, 8, 8, 1
        total_kv = k.shape[0]
    else:
        nb, nkv, bs, _ = _pool_geometry(k, layout)
        sb, sh, st = pool_strides(k, layout)
        mb = block_tables.shape[1]
        total_kv = int(kh[-1])
    if workspace is None:
        workspace = alloc_workspace(ragged_prefill_workspace_size(batch, total_qo, nq, hd),
                                    q.device)
    _check(load().pa_ragged_prefill(
        _ptr(o), _ptr(q), _ptr(k), _ptr(v), qh.ctypes.data_as(ctypes.c_void_p),
        kh.ctypes.data_as(ctypes.c_void_p), _ptr(qo_indptr_d), _ptr(kv_indptr_d),
        _ptr(block_tables), mb, bs, nb, sb, sh, st, batch, total_qo, total_kv, nq, nkv, hd,
        float(sm_scale), 1 if causal else 0, int(sliding_window), _ptr(workspace),
        workspace.numel(), _stream(stream)))


# The kernels take addresses: a tensor of another type, with gaps or on another device would be read
# as if it were what they expect.  The calls below look at every operand first, and read each
# property once (a short tree's call is as long as its kernel).
_INT32, _BF16 = torch.int32, torch.bfloat16


def _addresses(*tensors):
    """(device, data pointers...) of tensors on the current device, where the library launches."""
    devices = list(map(torch.Tensor.get_device, tensors))   # -1: not on a GPU
    device = devices[0]
    assert device >= 0 and devices.count(device) == len(devices) and \
        device == torch.cuda.current_device(), "tensors must be on the current CUDA device"
    return (device, *map(torch.Tensor.data_ptr, tensors))


def _check_int32(n, *arrays):
    for t in arrays:
        assert t.dtype is _INT32 and t.is_contiguous() and t.numel() >= n, \
            "tables, lengths and offsets must be dense int32 tensors that cover the batch"


def _kv_pools(k_cache, v_cache, layout):
    """(num_blocks, kv heads, block size, head_dim, strides of a block, head, token, kv_dtype)."""
    shape, strides, kind = k_cache.shape, k_cache.stride(), kv_dtype_of(k_cache)
    assert len(shape) == 4 and strides[3] == 1, "pool must be 4-D with a contiguous head_dim"
    assert v_cache.shape == shape and v_cache.stride() == strides and \
        (v_cache.dtype is k_cache.dtype or kv_dtype_of(v_cache) == kind), \
        "the K and V pools differ in geometry or type"
    nb, x, y, hd = shape
    sb, sx, sy, _ = strides
    return (nb, x, y, hd, sb, sx, sy, kind) if layout == "HND" else (nb, y, x, hd, sb, sy, sx, kind)


def _rows(out, q, head_dim):
    """(rows, query heads) of q, which out is to be like."""
    shape = q.shape
    rows, heads, hd = shape
    assert hd == head_dim and out.shape == shape and q.dtype is out.dtype is _BF16 and \
        q.is_contiguous() and out.is_contiguous(), \
        "q and out must be dense bf16 tensors of one shape, with the pools' head_dim"
    return rows, heads


def tree_decode_workspace_size(num_seqs, max_tree_len, num_q_heads, num_kv_heads, head_dim) -> int:
    return int(load().pa_tree_decode_workspace_size(num_seqs, max_tree_len, num_q_heads,
                                                    num_kv_heads, head_dim))


def pa_tree_decode(out, q, k_cache, v_cache, block_tables, seq_lens, qo_indptr, tree_mask, sm_scale,
                   max_tree_len, workspace, layout="HND", stream=None, sliding_window=0,
                   k_scale=1.0, v_scale=1.0):
    """Attention of drafted token trees into out [rows, nq, hd].  Sequence b's nodes are rows
    qo_indptr[b] .. qo_indptr[b + 1] - 1 of q and the last tokens of its cache (counted in
    seq_lens); each sees the context and the nodes whose bits tree_mask [rows, words] (int64)
    sets for it.  max_tree_len is at least the largest tree."""
    nb, nkv, bs, hd, sb, sh, st, kind = _kv_pools(k_cache, v_cache, layout)
    rows, nq = _rows(out, q, hd)
    mask_rows, words = tree_mask.shape
    seqs, blocks = block_tables.shape
    assert tree_mask.dtype == torch.int64 and tree_mask.is_contiguous() and mask_rows == rows, \
        "tree_mask must be a dense int64 tensor with a row of words per row of q"
    _check_int32(seqs, block_tables, seq_lens)
    _check_int32(seqs + 1, qo_indptr)
    assert workspace.is_contiguous(), "workspace must be dense"
    device, o, q, k, v, tables, lens, indptr, mask, ws = _addresses(
        out, q, k_cache, v_cache, block_tables, seq_lens, qo_indptr, tree_mask, workspace)
    _check(load().pa_tree_decode(o, q, k, v, tables, lens, indptr, mask, words, seqs, rows,
                                 int(max_tree_len), nq, nkv, hd, bs, blocks, nb, sb, sh, st,
                                 float(sm_scale), int(sliding_window), kind, float(k_scale),
                                 float(v_scale), ws, workspace.numel(), _stream(stream, device)))


def _all_pools(key_caches, value_caches, layout):
    """The pools of all layers in one list, of one geometry, and that geometry:
    (num_blocks, kv heads, block size, head_dim), strides of a block, head and token."""
    assert len(key_caches) == len(value_caches) > 0, "every layer has a key and a value pool"
    pools = [*key_caches, *value_caches]
    geometry = _pool_geometry(pools[0], layout), pool_strides(pools[0], layout)
    # a model has two pools a layer, so the checks go over whole lists
    n = len(pools)
    layouts = list(map(torch.Tensor.is_contiguous, pools))   # contiguous ones need no strides
    if not all(layouts):
        layouts = list(map(torch.Tensor.stride, pools))
    for values in ([t.shape for t in pools], layouts, [t.dtype for t in pools]):
        assert values.count(values[0]) == n, "pools differ in geometry"
    return pools, *geometry


def pa_tree_commit(key_caches, value_caches, block_tables, seq_lens, qo_indptr, accepted,
                   accept_lens, new_seq_lens, max_tree_len, layout="HND", stream=None):
    """Moves the K/V rows of each sequence's accepted nodes (accepted int32 [B, n], ascending,
    accept_lens[b] of them) behind its context in every layer's pools, and writes the
    sequences' new lengths into new_seq_lens (not seq_lens itself).  Layers that share a cache
    list it once."""
    pools, (nb, nkv, bs, hd), (sb, sh, st) = _all_pools(key_caches, value_caches, layout)
    seqs, blocks = block_tables.shape
    paths, most = accepted.shape
    assert accepted.dtype is _INT32 and accepted.is_contiguous() and paths >= seqs, \
        "accepted must be a dense int32 tensor with a row per sequence"
    _check_int32(seqs, block_tables, seq_lens, accept_lens, new_seq_lens)
    _check_int32(seqs + 1, qo_indptr)
    device, tables, lens, indptr, path, kept, new, *at = _addresses(
        block_tables, seq_lens, qo_indptr, accepted, accept_lens, new_seq_lens, *pools)
    at = array.array("Q", at)
    _check(load().pa_tree_commit(at.buffer_info()[0], len(pools), tables, lens, indptr, path, kept, new,
                                 seqs, int(max_tree_len), most, nkv, hd, bs, blocks, nb, sb, sh,
                                 st, kv_dtype_of(pools[0]), _stream(stream, device)))


def pa_page_bounds(bounds, k_cache, block_tables, seq_lens, max_new_tokens, first_tokens=None,
                   layout="HND", stream=None):
    """Rewrites bounds [num_blocks, nkv, 2, hd] (per-channel min and max of a page's keys, of the
    pool's type) for the pages that hold a token >= first_tokens[b] (None: every page);
    max_new_tokens is at least seq_lens[b] - first_tokens[b] for every sequence."""
    nb, nkv, bs, hd = _pool_geometry(k_cache, layout)
    sb, sh, st = pool_strides(k_cache, layout)
    seqs, blocks = block_tables.shape
    kind = kv_dtype_of(k_cache)
    assert bounds.is_contiguous() and bounds.shape == (nb, nkv, 2, hd) and \
        kv_dtype_of(bounds) == kind, \
        "bounds must be a dense [num_blocks, nkv, 2, hd] tensor of the pool's type"
    first = () if first_tokens is None else (first_tokens,)
    _check_int32(seqs, block_tables, seq_lens, *first)
    device, out, k, tables, lens, *first = _addresses(bounds, k_cache, block_tables, seq_lens,
                                                      *first)
    _check(load().pa_page_bounds(out, k, tables, lens, first[0] if first else None,
                                 int(max_new_tokens), seqs, nkv, hd, bs, blocks, nb, sb, sh, st,
                                 kind, _stream(stream, device)))


def select_pages_workspace_size(num_seqs, num_kv_heads, max_blocks_per_seq) -> int:
    return int(load().pa_select_pages_workspace_size(num_seqs, num_kv_heads, max_blocks_per_seq))


def pa_select_pages(page_tables, page_lens, q, bounds, block_tables, seq_lens, workspace,
                    sink_pages=0, recent_pages=1, stream=None):
    """Chooses up to max_pages pages per (sequence, kv head) for the queries q [B, nq, hd] by the
    pages' key bounds, into page_tables [B, nkv, max_pages] and page_lens [B] (int32); the
    first sink_pages and the last recent_pages are always among them."""
    nb, nkv, two, hd = bounds.shape
    B, nq, qd = q.shape
    rows, heads, most = page_tables.shape
    blocks = block_tables.shape[1]
    assert bounds.is_contiguous() and two == 2, "bounds must be dense, [num_blocks, nkv, 2, hd]"
    assert q.dtype is _BF16 and q.is_contiguous() and qd == hd, \
        "q must be a dense bf16 tensor with the bounds' head_dim"
    assert rows == B and heads == nkv, "page_tables must be [B, nkv, max_pages]"
    _check_int32(B, page_tables, page_lens, seq_lens)
    _check_int32(B * blocks, block_tables)
    assert workspace.is_contiguous(), "workspace must be dense"
    device, pages, kept, at, bnd, tables, lens, ws = _addresses(
        page_tables, page_lens, q, bounds, block_tables, seq_lens, workspace)
    _check(load().pa_select_pages(pages, kept, at, bnd, tables, lens, B, nq, nkv, hd, PAGE_TOKENS,
                                  blocks, nb, most, int(sink_pages), int(recent_pages),
                                  kv_dtype_of(bounds), ws, workspace.numel(),
                                  _stream(stream, device)))


def pa_decode_pages(out, q, k_cache, v_cache, page_tables, page_lens, sm_scale, workspace,
                    layout="HND", stream=None, k_scale=1.0, v_scale=1.0):
    """Split decode of q [B, nq, hd] over the pages page_tables [B, nkv, max_pages] lists per
    (sequence, kv head), page_lens[b] tokens each; the workspace is that of a split decode
    of max_pages pages."""
    nb, nkv, bs, hd, sb, sh, st, kind = _kv_pools(k_cache, v_cache, layout)
    B, nq = _rows(out, q, hd)
    rows, heads, most = page_tables.shape
    assert rows == B and heads == nkv, "page_tables must be [B, nkv, max_pages]"
    _check_int32(B, page_tables, page_lens)
    assert workspace.is_contiguous(), "workspace must be dense"
    device, o, q, k, v, tables, lens, ws = _addresses(out, q, k_cache, v_cache, page_tables,
                                                      page_lens, workspace)
    _check(load().pa_decode_pages(o, q, k, v, tables, lens, B, nq, nkv, hd, bs, most, nb, sb, sh,
                                  st, float(sm_scale), kind, float(k_scale), float(v_scale), ws,
                                  workspace.numel(), _stream(stream, device)))


ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}   # pa_rope_scaling
_LOW_HIGH = {"bands": (1.0, 4.0), "yarn": (1.0, 32.0)}


def rope_table(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_len=0, low=None,
               high=None, device="cuda"):
    """(turns, attention_factor) of the frequencies base^(-2 i / rotary_dim) under a scaling of
    ROPE_SCALINGS for long contexts: the int64 device table that pa_rope and pa_rope_append take,
    and the factor for their attention_factor.  low and high default to the usual 1 and 4 turns
    ("bands") or 1 and 32 ("yarn")."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling {scaling!r} is none of {sorted(ROPE_SCALINGS)}")
    usual = _LOW_HIGH.get(scaling, (1.0, 4.0))
    turns = torch.empty(max(0, int(rotary_dim) // 2), dtype=torch.int64)
    m = ctypes.c_float(1.0)
    _check(load().pa_rope_table(turns.data_ptr(), ctypes.addressof(m), int(rotary_dim), float(base),
                                ROPE_SCALINGS[scaling], float(factor),
                                float(usual[0] if low is None else low),
                                float(usual[1] if high is None else high), int(original_len)))
    return turns.to(device), m.value


def rope_table_of(frequencies, device="cuda"):
    """The table of any other frequencies (radians per position, one per pair)."""
    f = torch.as_tensor(frequencies, dtype=torch.float64).cpu().contiguous()
    turns = torch.empty(f.numel(), dtype=torch.int64)
    _check(load().pa_rope_table_of(turns.data_ptr(), f.data_ptr(), f.numel()))
    return turns.to(device)


_INT64 = torch.int64


_HEADS = "q, k, v and their outputs must be bf16 [tokens, heads, head_dim] of one token count and " \
    "head_dim, with a contiguous head_dim; q_out must be like q, k_out like k, k and v like the pools"
_PER_TOKEN = "positions, slots and frequencies must be dense int64 tensors, one entry a token or pair"


def _turned_rows(out, x, tokens, head_dim):
    """(heads, strides of a token and a head of out and of x), x [tokens, heads, head_dim]."""
    shape = x.shape
    t, heads, hd = shape
    out_token, out_head, out_step = out.stride()
    token, head, step = x.stride()
    assert x.dtype is out.dtype is _BF16 and out.shape == shape and t == tokens and hd == head_dim and \
        step == out_step == 1, _HEADS
    return heads, out_token, out_head, token, head


def _pairs_of(turns):
    n, = turns.shape
    assert turns.dtype is _INT64 and turns.is_contiguous(), _PER_TOKEN
    return n


def pa_rope(q_out, k_out, q, k, positions, turns, interleaved=False, attention_factor=1.0,
            inverse=False, stream=None):
    """q [T, nq, hd] and k [T, nk, hd] turned to positions [T] (int64) into q_out and k_out, which
    may be q and k themselves; k and k_out may be None.  turns and attention_factor are those of
    rope_table; the first 2 * len(turns) channels turn.  Slices of a fused projection are taken as
    they are.  inverse: by the negated angles, the gradient of the call without it."""
    t, _, hd = q.shape
    nq, qot, qoh, qt, qh = _turned_rows(q_out, q, t, hd)
    nk = kt = kh = kot = koh = 0
    more = ()
    assert (k is None) == (k_out is None), _HEADS
    if k is not None:
        nk, kot, koh, kt, kh = _turned_rows(k_out, k, t, hd)
        more = (k_out, k)
    pairs = _pairs_of(turns)
    assert positions.dtype is _INT64 and positions.shape == (t,) and positions.is_contiguous(), _PER_TOKEN
    device, qo, qi, pos, table, *more = _addresses(q_out, q, positions, turns, *more)
    ko, ki = more or (None, None)
    _check(load().pa_rope(qo, ko, qi, ki, pos, table, t, nq, nk, hd, 2 * pairs, qot, qoh, kot, koh, qt, qh,
                          kt, kh, 1 if interleaved else 0, 1 if inverse else 0, attention_factor,
                          _stream(stream, device)))


def pa_rope_append(q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, turns, layout="HND",
                   interleaved=False, attention_factor=1.0, stream=None, k_scale=1.0, v_scale=1.0):
    """pa_rope and pa_write_cache in one pass: q [T, nq, hd] turned into q_out, k [T, nkv, hd]
    turned into its slots of the cache, v into them as it is.  A token with a negative slot is
    padding and leaves its row of q_out as it was.  q and q_out may be None."""
    nb, nkv, bs, hd, sb, sh, st, kind = _kv_pools(k_cache, v_cache, layout)
    shape = k.shape
    t, heads, wide = shape
    kt, kh, step = k.stride()
    vt, vh, also = v.stride()
    assert heads == nkv and wide == hd and v.shape == shape and step == also == 1 and \
        k.dtype is v.dtype is _BF16 and (q is None) == (q_out is None), _HEADS
    nq = qt = qh = qot = qoh = 0
    more = ()
    if q is not None:
        nq, qot, qoh, qt, qh = _turned_rows(q_out, q, t, hd)
        more = (q_out, q)
    pairs = _pairs_of(turns)
    assert positions.dtype is slot_mapping.dtype is _INT64 and positions.shape == slot_mapping.shape == (t,) and \
        positions.is_contiguous() and slot_mapping.is_contiguous(), _PER_TOKEN
    device, ki, vi, kc, vc, slots, pos, table, *more = _addresses(k, v, k_cache, v_cache, slot_mapping,
                                                                  positions, turns, *more)
    qo, qi = more or (None, None)
    _check(load().pa_rope_append(qo, qi, ki, vi, kc, vc, slots, pos, table, t, nq, nkv, hd, 2 * pairs, bs, nb,
                                 qot, qoh, qt, qh, kt, kh, vt, vh, sb, sh, st, 1 if interleaved else 0,
                                 attention_factor, kind, k_scale, v_scale, _stream(stream, device)))


def beam_select_workspace_size(num_requests, num_beams, vocab) -> int:
    return int(load().pa_beam_select_workspace_size(num_requests, num_beams, vocab))


_LOGITS = {torch.float32: 0, torch.bfloat16: 1}   # pa_logits_dtype


def pa_beam_select(scores, beams, tokens, logits, cum_scores, workspace, finished=None, end_token=0,
                   stream=None):
    """The best pairs of beam and token of each request by cum_scores + log_softmax(logits), best
    first, into scores (float32), beams and tokens (int32), all [R, num_out].  logits [R * B, vocab]
    (float32 or bfloat16, rows any stride apart), cum_scores [R, B] (-inf: not in the search),
    finished [R, B] (uint8 or bool): those beams offer end_token at their score alone."""
    requests, num_beams = cum_scores.shape
    rows, vocab = logits.shape
    outs, num_out = scores.shape
    row_stride, one = logits.stride()
    assert logits.dtype in _LOGITS and rows == requests * num_beams and (one == 1 or vocab == 1), \
        "logits must be float32 or bfloat16 [requests * beams, vocab] with contiguous rows"
    assert cum_scores.dtype is scores.dtype is torch.float32 and cum_scores.is_contiguous() and \
        scores.is_contiguous() and outs == requests and beams.shape == tokens.shape == scores.shape, \
        "scores and cum_scores must be dense float32, scores, beams and tokens [requests, num_out]"
    _check_int32(outs * num_out, beams, tokens)
    assert workspace.is_contiguous(), "workspace must be dense"
    flags = ()
    if finished is not None:
        assert finished.dtype in (torch.uint8, torch.bool) and finished.is_contiguous() and \
            finished.shape == cum_scores.shape, "finished must be dense uint8 or bool, like cum_scores"
        flags = (finished,)
    device, sc, bm, tk, lg, cum, ws, *flags = _addresses(scores, beams, tokens, logits, cum_scores, workspace,
                                                         *flags)
    _check(load().pa_beam_select(sc, bm, tk, lg, cum, flags[0] if flags else None, int(end_token), requests,
                                 num_beams, vocab, num_out, row_stride, _LOGITS[logits.dtype], ws,
                                 workspace.numel() * workspace.element_size(), _stream(stream, device)))


def pa_beam_reorder(key_caches, value_caches, block_tables, seq_lens, parents, layout="HND",
                    stream=None):
    """The cache follows the chosen beams: sequence j of each request goes on from what sequence
    parents[r, j] (int32 [R, B]; -1: out of the search) held, in every layer's pools.  The full
    pages' ids move in block_tables [R * B, blocks] (in place), the rows of the page that the next
    token goes to, each sequence's own, are copied.  Layers that share a cache list it once."""
    pools, (nb, nkv, bs, hd), (sb, sh, st) = _all_pools(key_caches, value_caches, layout)
    requests, num_beams = parents.shape
    seqs, blocks = block_tables.shape
    assert seqs == requests * num_beams, "block_tables must have a row per request and beam"
    _check_int32(seqs, block_tables, seq_lens, parents)
    device, tables, lens, of, *at = _addresses(block_tables, seq_lens, parents, *pools)
    at = array.array("Q", at)
    _check(load().pa_beam_reorder(at.buffer_info()[0], len(pools), tables, lens, of, requests, num_beams,
                                  nkv, hd, bs, blocks, nb, sb, sh, st, kv_dtype_of(pools[0]),
                                  _stream(stream, device)))


def selftest_wait_timeout(stream=None):
    """Runs one bounded wait that nothing completes (about 1 s); the device status
    then holds the PA_ERR_TIMEOUT bit."""
    _check(load().pa_selftest_wait_timeout(_stream(stream)))


def device_status(stream=None) -> int:
    """Synchronise the stream, then read and clear the device status bits."""
    st = ctypes.c_int(0)
    _check(load().pa_get_device_status(ctypes.byref(st), _stream(stream)))
    return st.value
