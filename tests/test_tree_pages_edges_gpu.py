"""Edges of the tree and page-selection calls: lengths and page ids out of range where nothing is
ranked, bounds of pages that are never ranked, query groups split over several kernel groups, padded
pools, captured commits, tables of 2^27 pages, which kernel takes page lists."""
import math

import pytest
import torch

import paged_kv_gqa_15_gb300 as pa
from tests import ref64
from tests import test_fp8_trees_gpu as F
from tests import test_pages_gpu as P
from tests import test_tree_gpu as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOUNDS = 1 << pa.PA_ERR_DEVICE_BOUNDS


# ---- lengths and page ids out of range ------------------------------------------------------

def test_selection_of_every_page_flags_bad_pages():
    for most in (50, 64):                           # the table's width, and more than it
        c = P.make([800, 333], 4, 2, 64, 70)
        P.fill_bounds(c)
        P.check_select(c, most, 1, 1)
        assert pa.device_status() == 0
        for bad in (-3, c["k"].shape[0], 2 ** 31 - 1):
            c["table"][1, 20] = bad                 # the last page of sequence 1
            P.check_select(c, most, 1, 1)
            assert pa.device_status() == BOUNDS


def test_selection_of_every_page_of_one_sequence_flags_its_bad_page():
    c = P.make([800, 100], 4, 2, 64, 71)
    P.fill_bounds(c)
    c["table"][1, 2] = -1
    P.check_select(c, 12, 1, 1)                     # sequence 0's pages are ranked, sequence 1's are not
    assert pa.device_status() == BOUNDS


def test_selection_of_every_page_flags_a_length_past_the_table():
    c = P.make([800, 800], 4, 2, 64, 72)
    P.fill_bounds(c)
    c["lens"][1] = 801
    pages, lens = P.select(c, 50, 1, 1)
    assert pa.device_status() == BOUNDS
    assert lens.tolist() == [800, 800] and torch.equal(pages[1, 0], c["table"][1])


@pytest.mark.parametrize("fp8", [False, True])
def test_a_tree_whose_length_passes_its_table_is_skipped(fp8):
    """Its nodes would be tokens that the table does not hold: no row of it is written."""
    c = T.gpu(T.make([60, 64, 60], [4, 4, 4], 8, 2, 128, seed=15, fp8=fp8))
    good = T.call(c)
    assert pa.device_status() == 0
    for n in (65, 10 ** 6, 2 ** 31 - 1):
        c["lens"][1] = n
        got = T.call(c)
        assert pa.device_status() == BOUNDS
        assert torch.equal(got[:4], good[:4]) and torch.equal(got[8:], good[8:]) and bool((got[4:8] == 7).all())


def test_a_commit_whose_length_passes_its_table_is_skipped():
    c = T.gpu(T.make([60, 64], [4, 4], 8, 2, 128, seed=16))
    pools = [c["k"].clone(), c["v"].clone()]
    c["lens"][1] = 65
    new = T.run_commit(c, pools, torch.tensor([[3], [3]], dtype=torch.int32), torch.tensor([1, 1], dtype=torch.int32))
    assert pa.device_status() == BOUNDS and new.tolist() == [57, 65]
    want, _ = ref64.commit([c["k"], c["v"]], c["table"].cpu(), [60, 60], [0, 4, 8], torch.tensor([[3], [3]]), [1, 0])
    assert all(torch.equal(g.cpu().view(torch.uint8), w.view(torch.uint8)) for g, w in zip(pools, want))


# ---- bounds of pages that are never ranked --------------------------------------------------

@pytest.mark.parametrize("fp8,poison", [(False, math.nan), (False, math.inf), (False, 3e38), (True, math.nan), (True, 448.0)])
def test_bounds_of_pages_that_are_not_ranked_do_not_widen_the_border(fp8, poison):
    """A newest page's bounds may lag its rows, so that they may hold anything; nor are the first
    pages ranked.  Such bounds must not send every page through the scores in 64 bits: the
    workspace's place for those, its last part, stays as it was."""
    c = P.make([1600, 1440, 690], 4, 2, 64, 73, fp8)
    P.fill_bounds(c)
    for b, n in enumerate((100, 90, 44)):
        ids = c["table"][b, [0, 1, n - 3, n - 2, n - 1]].long()
        c["bounds"][ids] = torch.tensor(poison).to(c["bounds"].dtype).to(DEV)
    want = ref64.select(c["q"], c["bounds"], c["table"].cpu(), c["lens"].cpu(), 20, 2, 3)
    ws = pa.alloc_workspace(pa.select_pages_workspace_size(3, 2, c["table"].shape[1]), DEV)
    ws.fill_(171)
    pages, lens = P.select(c, 20, 2, 3, ws)
    assert torch.equal(pages.cpu(), want[0]) and torch.equal(lens.cpu(), want[1])
    assert bool((ws[-3 * 2 * 100 * 8:] == 171).all())
    assert pa.device_status() == 0


# ---- groups that are split ------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nq,nkv,lens,nodes", [(320, 2, [150, 90], [3, 2]), (393, 3, [70], [2])])
def test_trees_of_groups_beyond_a_row_tile(nq, nkv, lens, nodes, fp8):
    """Several kernel groups per kv head, each kv head with keys of its own."""
    c = T.gpu(T.make(lens, nodes, nq, nkv, 64, seed=74, fp8=fp8))
    T.check(c, T.call(c))
    assert pa.device_status() == 0


def test_values_that_are_not_finite_in_split_groups():
    """The values taken out of a tile are looked up again under the pool's kv head."""
    c = T.make([90], [4], 320, 2, 64, seed=75)
    for kh, node in ((0, 1), (1, 2)):
        c["v"][c["table"][0, (86 + node) // 16], kh, (86 + node) % 16] = math.inf
    c["mask"][:, 0] = torch.tensor([1, 2, 4, 8])
    got = T.call(T.gpu(c)).cpu()
    want = torch.zeros(4, 320, dtype=torch.bool)
    want[1, :160] = want[2, 160:] = True
    assert torch.equal(torch.isinf(got).all(-1), want) and torch.equal(torch.isfinite(got).all(-1), ~want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nq,nkv,hd", [(48, 2, 128), (24, 2, 128), (34, 2, 128), (51, 3, 128), (22, 2, 64), (6, 2, 256)])
def test_page_lists_of_split_groups(nq, nkv, hd, fp8):
    """Every kv head has a list of its own, also where its query heads are several kernel groups."""
    c = P.make([1500, 40, 977], nq, nkv, hd, 76, fp8)
    P.fill_bounds(c)
    pages, lens = P.check_select(c, 37, 1, 2)
    assert not torch.equal(pages[0, 0], pages[0, 1])
    out, bound = ref64.decode_pages(c["q"], c["k"], c["v"], pages.cpu(), lens.cpu(), c["scale"], "HND", c["kv_scale"],
                                    c["kv_scale"])
    ref64.assert_attention(P.decode(c, pages, lens), out, bound, P.FP8_EXTRA if fp8 else 0.0)
    assert pa.device_status() == 0


# ---- which kernel takes page lists ----------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nq,nkv,hd", [(4, 1, 256), (6, 1, 256), (14, 2, 256), (24, 2, 256), (9, 1, 64), (24, 2, 64),
                                       (16, 1, 64)])
def test_few_pages_are_the_split_decode_for_wide_groups_too(nq, nkv, hd, fp8):
    """The tree kernel takes longer there (a list is a chain of tiles), so all pages of short sequences
    give the split decode's bits."""
    c = P.make([900, 40, 477], nq, nkv, hd, 81, fp8)
    P.fill_bounds(c)
    pages, lens = P.select(c, 57, 0, 1)
    ws = pa.alloc_workspace(pa.decode_split_workspace_size(3, nq, hd, 57 * 16), DEV)
    want = torch.empty_like(c["q"])
    pa.pa_decode_split(want, c["q"], c["k"], c["v"], c["table"], c["lens"], c["scale"], 57 * 16, ws, k_scale=c["kv_scale"],
                       v_scale=c["kv_scale"])
    assert torch.equal(P.decode(c, pages, lens), want)
    assert pa.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nq,nkv,hd,seqs,most", [(9, 1, 64, 24, 290), (24, 2, 64, 18, 190), (11, 1, 64, 3, 640), (3, 1, 64, 30, 230),
                                                 (16, 2, 256, 3, 70), (3, 1, 256, 20, 180), (10, 2, 256, 12, 70),
                                                 (12, 3, 256, 9, 190), (9, 1, 64, 60, 8), (12, 2, 256, 30, 31)])
def test_many_pages_of_wide_groups(nq, nkv, hd, seqs, most, fp8):
    """Enough reading for the tree kernel, in whole and in cut runs; every kv head's list is its own."""
    lens = [most * 16 + 700 - 37 * (i % 19) for i in range(seqs - 2)] + [0, 33]
    c = P.make(lens, nq, nkv, hd, 82, fp8)
    gen = torch.Generator().manual_seed(5)
    pages = torch.stack([torch.stack([torch.randperm(c["k"].shape[0] - 3, generator=gen)[:most] for _ in range(nkv)])
                         for _ in lens]).int()
    c["k"], c["v"] = (x.float().nan_to_num(0.0).to(x.dtype) for x in (c["k"], c["v"]))
    kept = torch.tensor([min(n, most * 16 - 5 * (i % 4)) for i, n in enumerate(lens)], dtype=torch.int32)
    got = P.decode(c, pages.to(DEV), kept.to(DEV))
    out, bound = ref64.decode_pages(c["q"], c["k"], c["v"], pages, kept, c["scale"], "HND", c["kv_scale"], c["kv_scale"])
    ref64.assert_attention(got, out, bound, F.extra(c["q"], c["k"], c["scale"], c["kv_scale"], most * 16) if fp8 else 0.0)
    assert bool((got[-2] == 0).all()) and torch.equal(P.decode(c, pages.to(DEV), kept.to(DEV)), got)
    assert pa.device_status() == 0


# ---- padded pools ---------------------------------------------------------------------------

def padded(pool):
    """The pool's values with room between pages, heads and tokens; codes of NaN in the room."""
    n, h, t, d = pool.shape
    raw = pool.view(torch.uint8)
    wide = torch.full((n, h + 1, t, d + 16), math.nan).to(pool.dtype).to(pool.device)
    view = wide[:, :h, :, :d]
    view.copy_(pool) if pool.dtype == torch.bfloat16 else view.view(torch.uint8).copy_(raw)
    return wide, view


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_commit_in_padded_pools(layout, fp8):
    c = T.gpu(T.make([40, 23], [12, 23], 4, 2, 64, seed=77, fp8=fp8, layout=layout))
    paths, kept = torch.tensor([[0, 3, 4, 11], [2, 5, 21, 22]], dtype=torch.int32), torch.tensor([4, 3], dtype=torch.int32)
    want, lens = ref64.commit([c["k"], c["v"]], c["table"].cpu(), c["lens"].cpu(), c["indptr"].cpu(), paths, kept, layout)
    whole, pools = zip(*(padded(c[n]) for n in ("k", "v")))
    before = [w.view(torch.uint8).clone() for w in whole]
    assert T.run_commit(c, list(pools), paths, kept).tolist() == lens
    for got, ref, w, b in zip(pools, want, whole, before):
        assert torch.equal(got.contiguous().cpu().view(torch.uint8), ref.view(torch.uint8))
        outside = torch.ones(w.shape, dtype=torch.bool, device=DEV)
        outside[:, :got.shape[1], :, :got.shape[3]] = False
        now = w.view(torch.uint8)
        if now.shape != w.shape:
            outside = outside.repeat_interleave(2, -1)
        assert torch.equal(now[outside], b[outside])
    assert pa.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("nq,nkv,hd", [(2, 2, 64), (8, 2, 128), (4, 1, 64), (16, 2, 256), (24, 2, 64)])
def test_bounds_and_page_lists_over_padded_pools(nq, nkv, hd, layout, fp8):
    c = P.make([700, 40], nq, nkv, hd, 78, fp8, layout)
    P.fill_bounds(c)
    dense = c["bounds"].clone()
    pages, lens = P.check_select(c, 17, 1, 2)
    want = P.decode(c, pages, lens)
    c["k"], c["v"] = padded(c["k"])[1], padded(c["v"])[1]
    c["bounds"].zero_()
    P.fill_bounds(c)
    assert torch.equal(c["bounds"].view(torch.uint8), dense.view(torch.uint8))
    assert torch.equal(P.decode(c, pages, lens), want)
    assert pa.device_status() == 0


# ---- capture --------------------------------------------------------------------------------

def test_a_captured_step_of_trees_and_commit_replays():
    """Verification and commit of all layers as one graph, replayed with other paths and trees."""
    c = T.gpu(T.make([100, 61], [6, 6], 8, 2, 128, seed=79))
    c["k"], c["v"] = c["k"].nan_to_num(0.0), c["v"].nan_to_num(0.0)
    keys, vals = [c["k"].clone() for _ in range(3)], [c["v"].clone() for _ in range(3)]
    path, kept = torch.tensor([[0, 2, 5], [1, 3, 0]], dtype=torch.int32, device=DEV), torch.tensor([3, 2], dtype=torch.int32, device=DEV)
    new, out, ws = torch.zeros(2, dtype=torch.int32, device=DEV), torch.full_like(c["q"], 7.0), T.space(c)

    def step():
        T.call(c, out=out, ws=ws)
        pa.pa_tree_commit(keys, vals, c["table"], c["lens"], c["indptr"], path, kept, new, 6)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for paths, n in (([[1, 2, 4], [0, 4, 5]], [3, 3]), ([[5, 0, 0], [2, 3, 4]], [1, 0]), ([[3, 4, 5], [3, 0, 0]], [3, 1])):
        path.copy_(torch.tensor(paths)), kept.copy_(torch.tensor(n))
        for i in range(3):
            keys[i].copy_(c["k"] + i), vals[i].copy_(c["v"] - i)
        pools = [t for kv in zip(keys, vals) for t in kv]
        want, lens = ref64.commit(pools, c["table"].cpu(), c["lens"].cpu(), c["indptr"].cpu(), path.cpu(), kept.cpu())
        graph.replay()
        torch.cuda.synchronize()
        T.check(c, out)
        assert new.tolist() == lens
        assert all(torch.equal(g.cpu().view(torch.uint8), w.view(torch.uint8)) for g, w in zip(pools, want))
    assert pa.device_status() == 0


# ---- the longest table ----------------------------------------------------------------------

def test_a_tree_behind_as_many_tokens_as_a_table_can_hold():
    """2^31 - 16 tokens in 2^27 - 1 pages, three pages over and over: the softmax over their 48 rows,
    weighted by how often each comes.  A CTA adds up 2^25 / 304 tiles in four products each, in fp32, each
    sum off by at most one step (2^-23); the sum of the weights, over two adds a tile and thread, by
    half as much: 0.053 + 0.027 of sum p |v|."""
    n_pages, nodes = (1 << 27) - 1, 3
    n = n_pages * 16
    c = T.make([48], [nodes], 2, 1, 64, seed=80)
    pages = c["table"][0, :3].clone()
    order = torch.arange(n_pages, dtype=torch.int32, device=DEV).remainder_(3)
    c = T.gpu(c)
    small = c["table"][0, :3].cpu().long()
    c["table"] = pages.to(DEV)[order.long()].view(1, -1).contiguous()
    c["lens"] = torch.tensor([n], dtype=torch.int32, device=DEV)
    got = T.call(c)
    assert pa.device_status() == 0
    last = (n_pages - 1) % 3
    times = torch.tensor([[(n_pages - p + 2) // 3] for p in range(3)], dtype=torch.float64).expand(3, 16).clone()
    times[last, 13:] -= 1                               # the nodes: rows 13 to 15 of the last page
    k, v = (c[x].cpu().double()[small, 0].flatten(0, 1) for x in ("k", "v"))
    out, bound = torch.zeros(nodes, 2, 64, dtype=torch.float64), torch.zeros(nodes, 2, 64, dtype=torch.float64)
    for i in range(nodes):
        w = times.clone()
        for j in ref64.mask_bits(c["mask"][i].cpu(), nodes):
            w[last, 13 + j] += 1
        for h in range(2):
            x = c["q"][i, h].cpu().double() @ k.T * c["scale"]
            p = torch.exp(x - x.max()) * w.flatten()
            p /= p.sum()
            out[i, h], bound[i, h] = p @ v, p @ v.abs()
    ref64.assert_attention(got, out, bound, extra=0.08)
