"""Host-side refusals of the tree and page-selection entry points (no GPU: validation comes before any
CUDA call): outputs that share memory with what the kernels still read."""
import ctypes

import pytest

import paged_kv_gqa_15_gb300 as pa


def at(i):
    """Buffers far from one another."""
    return 0x1000000 * (i + 1)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return pa.load()


def commit(lib, **kw):
    a = dict(pools=(ctypes.c_void_p * 2)(at(0), at(1)), bt=at(2), sl=at(3), ip=at(4), acc=at(5), al=at(6),
             new=at(7), B=8, A=4, mb=4)
    a.update(kw)
    code = lib.pa_tree_commit(a["pools"], 2, a["bt"], a["sl"], a["ip"], a["acc"], a["al"], a["new"], a["B"], 8, a["A"],
                              2, 128, 16, a["mb"], 10, 4096, 2048, 128, 0, None)
    return code, lib.pa_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(new=at(5)), dict(new=at(5) + 8 * 4 * 4 - 4), dict(new=at(5) - 8 * 4 + 4),   # accepted
    dict(new=at(2)), dict(new=at(2) + 8 * 4 * 4 - 4), dict(new=at(2) - 8 * 4 + 4),   # block_tables
    dict(new=at(3)), dict(new=at(4) + 8 * 4), dict(new=at(6)),
])
def test_new_lengths_over_what_the_commit_reads(lib, kw):
    code, why = commit(lib, **kw)
    assert code == pa.PA_ERR_INVALID and "new_seq_lens" in why


def select(lib, **kw):
    a = dict(pt=at(0), pl=at(1), bt=at(2), sl=at(3), B=8, nkv=2, most=4, mb=8)
    a.update(kw)
    code = lib.pa_select_pages(a["pt"], a["pl"], at(4), at(5), a["bt"], a["sl"], a["B"], 8, a["nkv"], 128, 16, a["mb"], 10,
                               a["most"], 1, 1, 0, at(6), 1 << 40, None)
    return code, lib.pa_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(pl=at(2)), dict(pl=at(2) + 8 * 8 * 4 - 4), dict(pl=at(2) - 8 * 4 + 4),      # page_lens, block_tables
    dict(pt=at(3)), dict(pt=at(3) + 8 * 4 - 4), dict(pt=at(3) - 8 * 2 * 4 * 4 + 4),  # page_tables, seq_lens
    dict(pt=at(1)), dict(pl=at(0) + 8 * 2 * 4 * 4 - 4),                              # one another
    dict(pl=at(3)), dict(pt=at(2)),
])
def test_page_lists_over_what_the_selection_reads(lib, kw):
    code, why = select(lib, **kw)
    assert code == pa.PA_ERR_INVALID and "page_lens and page_tables" in why


@pytest.mark.parametrize("nkv,blocks,new,code", [
    (17, (1 << 27) - 1, 2 ** 31 - 1, pa.PA_ERR_UNSUPPORTED),      # a sequence's (page, head) pairs pass 2^31
    (128, (1 << 27) - 1, 2 ** 31 - 1, pa.PA_ERR_UNSUPPORTED),
    (1 << 20, 1 << 12, 1 << 16, pa.PA_ERR_UNSUPPORTED),
])
def test_bounds_of_more_pages_than_32_bits_count(lib, nkv, blocks, new, code):
    assert lib.pa_page_bounds(at(0), at(1), at(2), at(3), None, new, 1, nkv, 64, 16, blocks, 10, 16 * nkv * 64, 1024, 64, 0,
                              None) == code
