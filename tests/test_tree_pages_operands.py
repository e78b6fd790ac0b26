"""The bindings of the tree and page-selection calls refuse operands that the kernels, which take
addresses alone, would misread: other types, shapes or devices, gaps between elements.

No GPU is needed: the operands are host tensors, the checks of a well-formed call end at the device."""
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa

NB, NKV, HD, NQ, B, ROWS = 6, 2, 64, 4, 3, 5


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return pa.load()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def pool(dtype=torch.bfloat16):
    return torch.zeros((NB, NKV, 16, HD), dtype=dtype)


def rows(n=ROWS):
    return torch.zeros((n, NQ, HD), dtype=torch.bfloat16)


def space():
    return torch.zeros(1 << 22, dtype=torch.uint8)


def tree(**kw):
    a = dict(out=rows(), q=rows(), k_cache=pool(), v_cache=pool(), block_tables=i32(B, 4), seq_lens=i32(B),
             qo_indptr=i32(B + 1), tree_mask=torch.zeros((ROWS, 1), dtype=torch.int64), sm_scale=1.0,
             max_tree_len=3, workspace=space())
    a.update(kw)
    pa.pa_tree_decode(**a)


def commit(**kw):
    a = dict(key_caches=[pool(), pool()], value_caches=[pool(), pool()], block_tables=i32(B, 4), seq_lens=i32(B),
             qo_indptr=i32(B + 1), accepted=i32(B, 2), accept_lens=i32(B), new_seq_lens=i32(B), max_tree_len=3)
    a.update(kw)
    pa.pa_tree_commit(**a)


def bounds(**kw):
    a = dict(bounds=torch.zeros((NB, NKV, 2, HD), dtype=torch.bfloat16), k_cache=pool(), block_tables=i32(B, 4),
             seq_lens=i32(B), max_new_tokens=3, first_tokens=i32(B))
    a.update(kw)
    pa.pa_page_bounds(**a)


def select(**kw):
    a = dict(page_tables=i32(B, NKV, 2), page_lens=i32(B), q=rows(B),
             bounds=torch.zeros((NB, NKV, 2, HD), dtype=torch.bfloat16), block_tables=i32(B, 4), seq_lens=i32(B),
             workspace=space())
    a.update(kw)
    pa.pa_select_pages(**a)


def pages(**kw):
    a = dict(out=rows(B), q=rows(B), k_cache=pool(), v_cache=pool(), page_tables=i32(B, NKV, 2), page_lens=i32(B),
             sm_scale=1.0, workspace=space())
    a.update(kw)
    pa.pa_decode_pages(**a)


def wide(t):
    """t's values with room between its rows, as a slice of a fused projection has."""
    return torch.cat([t, t], -1)[..., :t.shape[-1]]


CALLS = [tree, commit, bounds, select, pages]


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors(call):
    with pytest.raises(AssertionError, match="current CUDA device"):
        call()


@pytest.mark.parametrize("call", CALLS)
def test_one_host_tensor_among_device_tensors(call, monkeypatch):
    """Every tensor of a call is looked at: all claim a device but one at a time."""
    class Library:              # nothing is launched
        def __getattr__(self, name):
            return lambda *args: pa.PA_OK
    monkeypatch.setattr(pa, "load", Library)
    monkeypatch.setattr(pa, "_stream", lambda *args: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    seen = []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: seen.append(t) or 0)
    call()
    n = len({id(t) for t in seen})
    assert n == {tree: 9, commit: 10, bounds: 5, select: 7, pages: 7}[call]
    n = len(seen)
    for at in range(n):
        seen = []
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: seen.append(t) or (-1 if len(seen) == at + 1 else 0))
        with pytest.raises(AssertionError, match="current CUDA device"):
            call()
        assert len(seen) > at
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    with pytest.raises(AssertionError, match="current CUDA device"):
        call()


@pytest.mark.parametrize("call,kw,what", [
    (tree, dict(q=wide(rows())), "q and out"),                       # a slice of a fused projection
    (tree, dict(q=rows().transpose(0, 1).contiguous().transpose(0, 1)), "q and out"),
    (tree, dict(q=rows().float()), "q and out"),
    (tree, dict(q=rows().half()), "q and out"),
    (tree, dict(out=rows().half()), "q and out"),
    (tree, dict(out=wide(rows())), "q and out"),
    (tree, dict(out=rows(ROWS - 1)), "q and out"),
    (tree, dict(q=torch.zeros((ROWS, NQ, 128), dtype=torch.bfloat16),
                out=torch.zeros((ROWS, NQ, 128), dtype=torch.bfloat16)), "q and out"),   # not the pools' head_dim
    (tree, dict(v_cache=pool()[:-1]), "pools"),
    (tree, dict(v_cache=wide(pool())), "pools"),
    (tree, dict(v_cache=pool(torch.uint8)), "pools"),
    (tree, dict(block_tables=wide(i32(B, 4))), "int32"),
    (tree, dict(block_tables=i32(B, 4).long()), "int32"),
    (tree, dict(seq_lens=i32(B).long()), "int32"),
    (tree, dict(seq_lens=i32(2 * B)[::2]), "int32"),
    (tree, dict(seq_lens=i32(B - 1)), "int32"),
    (tree, dict(qo_indptr=i32(B + 1).long()), "int32"),
    (tree, dict(qo_indptr=i32(B)), "int32"),
    (tree, dict(tree_mask=torch.zeros((ROWS, 2), dtype=torch.int64)[:, :1]), "tree_mask"),
    (tree, dict(tree_mask=torch.zeros((ROWS - 1, 1), dtype=torch.int64)), "tree_mask"),
    (tree, dict(workspace=space()[::2]), "workspace"),
    (commit, dict(block_tables=wide(i32(B, 4))), "int32"),
    (commit, dict(block_tables=i32(B, 4).long()), "int32"),
    (commit, dict(seq_lens=i32(B).long()), "int32"),
    (commit, dict(seq_lens=i32(B - 1)), "int32"),
    (commit, dict(qo_indptr=i32(B)), "int32"),
    (commit, dict(accept_lens=i32(B).long()), "int32"),
    (commit, dict(accept_lens=i32(B - 1)), "int32"),
    (commit, dict(new_seq_lens=i32(B).long()), "int32"),
    (commit, dict(new_seq_lens=i32(B - 1)), "int32"),
    (commit, dict(new_seq_lens=i32(2 * B)[::2]), "int32"),
    (commit, dict(accepted=i32(B - 1, 2)), "accepted"),
    (commit, dict(accepted=wide(i32(B, 2))), "accepted"),
    (commit, dict(value_caches=[pool(), wide(pool())]), "pools"),
    (bounds, dict(bounds=torch.zeros((NB, NKV, 2, HD), dtype=torch.uint8)), "bounds"),
    (bounds, dict(bounds=wide(torch.zeros((NB, NKV, 2, HD), dtype=torch.bfloat16))), "bounds"),
    (bounds, dict(block_tables=wide(i32(B, 4))), "int32"),
    (bounds, dict(seq_lens=i32(B).long()), "int32"),
    (bounds, dict(seq_lens=i32(B - 1)), "int32"),
    (bounds, dict(first_tokens=i32(B).long()), "int32"),
    (bounds, dict(first_tokens=i32(B - 1)), "int32"),
    (select, dict(q=wide(rows(B))), "q must"),
    (select, dict(q=rows(B).half()), "q must"),
    (select, dict(q=torch.zeros((B, NQ, 128), dtype=torch.bfloat16)), "q must"),
    (select, dict(bounds=wide(torch.zeros((NB, NKV, 2, HD), dtype=torch.bfloat16))), "bounds"),
    (select, dict(bounds=torch.zeros((NB, NKV, 1, HD), dtype=torch.bfloat16)), "bounds"),
    (select, dict(block_tables=wide(i32(B, 4))), "int32"),
    (select, dict(block_tables=i32(B - 1, 4)), "int32"),
    (select, dict(seq_lens=i32(B).long()), "int32"),
    (select, dict(seq_lens=i32(B - 1)), "int32"),
    (select, dict(page_tables=i32(B, NKV, 2).long()), "int32"),
    (select, dict(page_tables=wide(i32(B, NKV, 2))), "int32"),
    (select, dict(page_lens=i32(B).long()), "int32"),
    (select, dict(page_lens=i32(B - 1)), "int32"),
    (select, dict(workspace=space()[::2]), "workspace"),
    (pages, dict(q=wide(rows(B))), "q and out"),
    (pages, dict(q=rows(B).half()), "q and out"),
    (pages, dict(out=rows(B).half()), "q and out"),
    (pages, dict(out=rows(B - 1)), "q and out"),
    (pages, dict(q=torch.zeros((B, NQ, 128), dtype=torch.bfloat16),
                 out=torch.zeros((B, NQ, 128), dtype=torch.bfloat16)), "q and out"),
    (pages, dict(v_cache=pool()[:-1]), "pools"),
    (pages, dict(v_cache=wide(pool())), "pools"),
    (pages, dict(v_cache=pool(torch.uint8)), "pools"),
    (pages, dict(page_tables=i32(B, NKV, 2).long()), "int32"),
    (pages, dict(page_tables=wide(i32(B, NKV, 2))), "int32"),
    (pages, dict(page_lens=i32(B).long()), "int32"),
    (pages, dict(page_lens=i32(B - 1)), "int32"),
    (pages, dict(workspace=space()[::2]), "workspace"),
])
def test_operands_the_kernels_would_misread(call, kw, what):
    with pytest.raises(AssertionError, match=what):
        call(**kw)


@pytest.mark.parametrize("call,kw", [
    (tree, dict(k_cache=pool(torch.uint8), v_cache=pool(torch.uint8).view(torch.float8_e4m3fn))),
    (tree, dict(k_cache=wide(pool()), v_cache=wide(pool()))),                    # padded pools
    (tree, dict(seq_lens=i32(B + 5), qo_indptr=i32(B + 6))),                     # buffers of a larger batch
    (commit, dict(key_caches=[wide(pool())], value_caches=[wide(pool())])),
    (commit, dict(accepted=i32(B + 4, 2), accept_lens=i32(B + 4), new_seq_lens=i32(B + 4))),
    (bounds, dict(first_tokens=None)),
    (bounds, dict(k_cache=pool(torch.uint8), bounds=torch.zeros((NB, NKV, 2, HD), dtype=torch.float8_e4m3fn))),
    (pages, dict(k_cache=pool(torch.uint8), v_cache=pool(torch.uint8).view(torch.float8_e4m3fn))),
    (pages, dict(k_cache=wide(pool()), v_cache=wide(pool()))),
])
def test_operands_that_are_as_good(call, kw):
    """Everything but the device passes."""
    with pytest.raises(AssertionError, match="current CUDA device"):
        call(**kw)
