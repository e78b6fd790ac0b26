"""Tree attention (pa_tree_decode) and path commit (pa_tree_commit) against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa
from tests import ref64

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAGE = 16


def make(lens, nodes, nq, nkv, hd, seed, fp8=False, layout="HND", pad_rows=0, words=None, shape="tree"):
    """Pools whose unused rows hold NaN, random trees, and q with `pad_rows` extra rows."""
    rng = np.random.default_rng(seed)
    need = [(n + PAGE - 1) // PAGE for n in lens]
    nb = sum(need) + 3
    perm = rng.permutation(nb)
    table = np.full((len(lens), max(max(need), 1)), np.iinfo(np.int32).max, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    gen = torch.Generator().manual_seed(seed)
    dims = (nb, nkv, PAGE, hd) if layout == "HND" else (nb, PAGE, nkv, hd)
    scale = 1.0 / 32 if fp8 else 1.0
    pools = []
    for _ in range(2):
        x = torch.full(dims, math.nan)
        for b, n in enumerate(lens):
            for t in range(n):
                row = torch.randn(nkv, hd, generator=gen)
                if layout == "HND":
                    x[table[b, t // PAGE], :, t % PAGE] = row
                else:
                    x[table[b, t // PAGE], t % PAGE] = row
        pools.append((x / scale).to(torch.float8_e4m3fn) if fp8 else x.to(torch.bfloat16))
    indptr = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    rows = int(indptr[-1]) + pad_rows
    words = words or (max(max(nodes), 1) + 63) // 64
    mask = np.zeros((rows, words), np.uint64)
    for b, n in enumerate(nodes):
        seen = []
        for i in range(n):
            parent = int(rng.integers(max(-1, i - 5), i)) if i else -1
            bits = (seen[parent] if parent >= 0 else 0) | 1 << i
            seen.append(bits)
            if shape == "any":      # not a tree: any subset, also none and bits past the tree
                bits = int(rng.integers(0, 2 ** 62)) if i % 3 else 0
            for w in range(words):
                mask[indptr[b] + i, w] = bits >> 64 * w & 0xFFFFFFFFFFFFFFFF
    q = torch.randn(rows, nq, hd, generator=gen).to(torch.bfloat16)
    return dict(q=q, k=pools[0], v=pools[1], table=torch.from_numpy(table),
                lens=torch.tensor(lens, dtype=torch.int32), indptr=torch.from_numpy(indptr),
                mask=torch.from_numpy(mask.view(np.int64)), kv_scale=scale, layout=layout,
                nodes=max(max(nodes), 1), scale=1.0 / math.sqrt(hd))


def gpu(c):
    return {n: v.to(DEV) if isinstance(v, torch.Tensor) else v for n, v in c.items()}


def space(c, extra=0):
    nkv = c["k"].shape[1 if c["layout"] == "HND" else 2]
    return pa.alloc_workspace(pa.tree_decode_workspace_size(
        len(c["lens"]), c["nodes"], c["q"].shape[1], nkv, c["q"].shape[2]) + extra, DEV)


def call(c, window=0, out=None, ws=None, stream=None):
    out = torch.full_like(c["q"], 7.0) if out is None else out
    pa.pa_tree_decode(out, c["q"], c["k"], c["v"], c["table"], c["lens"], c["indptr"], c["mask"],
                      c["scale"], c["nodes"], space(c) if ws is None else ws, layout=c["layout"],
                      sliding_window=window, k_scale=c["kv_scale"], v_scale=c["kv_scale"],
                      stream=stream)
    return out


# An 8-bit cache's scores: q as the sum of E4M3 values to 2^-8 of its value moves a score by at
# most 2^-8 sum |q k| scale (under 16 for these inputs), a weight by a factor 1 +- 0.065, and
# the normalisation by as much; the weights themselves by 2^-8 of theirs and 2^-18 of the largest.
FP8_EXTRA = 0.14


def check(c, got, window=0, what=""):
    rows = int(c["indptr"][-1])
    fp8 = c["k"].dtype != torch.bfloat16
    out, bound = ref64.tree(c["q"][:rows].cpu(), c["k"], c["v"], c["table"].cpu(), c["lens"].cpu(),
                            c["indptr"].cpu(), c["mask"].cpu(), c["scale"], c["layout"], window,
                            c["kv_scale"], c["kv_scale"])
    ref64.assert_attention(got[:rows], out, bound, FP8_EXTRA if fp8 else 0.0, what)
    assert bool((got[rows:] == 7.0).all()), "rows behind the last sequence were written"


CASES = [
    # lens, nodes, nq, nkv, hd
    ([1], [1], 1, 1, 64),
    ([5, 40], [5, 3], 4, 2, 64),
    ([17, 33, 64, 100], [1, 8, 16, 7], 4, 2, 64),
    ([130, 1, 700], [16, 1, 9], 8, 2, 128),
    ([64, 65, 128, 129], [4, 4, 4, 4], 12, 4, 128),
    ([600, 31], [40, 31], 14, 2, 128),
    ([90], [33], 5, 1, 128),
    ([300, 20, 77], [21, 5, 1], 6, 3, 256),
    ([260], [17], 16, 1, 256),
    ([220, 300], [200, 130], 4, 2, 64),
    ([1300], [60], 32, 8, 128),
    ([150], [3], 40, 2, 128),
    ([70, 50], [2, 1], 71, 1, 64),
    ([90], [2], 160, 1, 64),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_tree_matches_64_bits(i, fp8):
    lens, nodes, nq, nkv, hd = CASES[i]
    c = gpu(make(lens, nodes, nq, nkv, hd, seed=100 + i, fp8=fp8, layout="NHD" if i % 2 else "HND",
                 pad_rows=i % 3))
    check(c, call(c), what=str(CASES[i]))
    assert pa.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [1, 5, 16, 33, 100, 1000])
def test_tree_under_a_sliding_window(window, fp8):
    c = gpu(make([300, 45, 129], [9, 20, 1], 8, 2, 128, seed=7, fp8=fp8))
    c["mask"][4] = 0                      # a row that sees no node
    check(c, call(c, window=window), window, f"window {window}")
    assert pa.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_masks_that_are_not_trees(fp8):
    """Any subset of nodes, rows that see none (with no context: zeros), bits past the tree."""
    for hd in (64, 128, 256):
        c = gpu(make([12, 12, 400, 62], [12, 7, 50, 62], 8, 4, hd, seed=hd, fp8=fp8, shape="any", words=2))
        got = call(c)
        check(c, got)
        assert bool((got[0] == 0).all())          # node 0 sees nothing and there is no context
    assert pa.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_that_all_but_vanish(fp8):
    """q of about 2^-120 and a scale of 2^-40: every weight is the same, and a row without a key
    in a tile, or in any, stays a number."""
    c = make([12, 200], [12, 100], 4, 2, 64, seed=31, fp8=fp8, shape="any")
    c["q"] *= 2.0 ** -120
    c["scale"] = 2.0 ** -40
    check(gpu(c), call(gpu(c)))
    assert pa.device_status() == 0


def test_unseen_nodes_and_stale_rows_may_hold_nan():
    c = make([70, 33], [8, 8], 8, 2, 128, seed=11)
    c["mask"][3] = 1 << 3
    for pool in (c["k"], c["v"]):                  # node 5 of sequence 0, seen by no other row
        pool[c["table"][0, (62 + 5) // PAGE], :, (62 + 5) % PAGE] = math.nan
    c["mask"][:8] &= ~(1 << 5)
    c = gpu(c)
    check(c, call(c))


def test_nan_and_infinite_keys_that_are_seen_reach_only_the_rows_that_see_them():
    c = make([80], [4], 4, 1, 128, seed=12)
    c["v"][c["table"][0, 78 // PAGE], :, 78 % PAGE] = math.nan   # node 2
    c["mask"][:, 0] = torch.tensor([1, 2, 4, 8])
    c = gpu(c)
    got = call(c).cpu()
    assert torch.isnan(got[2]).all()
    out, bound = ref64.tree(c["q"], c["k"], c["v"], c["table"].cpu(), c["lens"].cpu(), c["indptr"].cpu(),
                            c["mask"].cpu(), c["scale"])
    keep = torch.tensor([0, 1, 3])
    ref64.assert_attention(got[keep], out[keep], bound[keep])


def test_large_scores():
    c = make([500], [16], 8, 2, 128, seed=13)
    c["q"] *= 40
    c = gpu(c)
    got = call(c)
    out, bound = ref64.tree(c["q"], c["k"], c["v"], c["table"].cpu(), c["lens"].cpu(), c["indptr"].cpu(),
                            c["mask"].cpu(), c["scale"])
    # scores up to 40 times larger: the fp32 score error grows with them (2.1e-3 * 40)
    ref64.assert_attention(got, out, bound, extra=0.084)


@pytest.mark.parametrize("fp8", [False, True])
def test_weights_far_under_one_large_maximum(fp8):
    """One key ten units above 4999 equal ones, which hold a fifth of the sum between them.  The
    scores are exact in every type (one channel, small whole numbers), so an 8-bit cache keeps
    the bounds of a bf16 one."""
    hd, n = 128, 5000
    c = make([n], [2], 4, 2, hd, seed=40, fp8=fp8)
    dt = c["k"].dtype
    c["scale"], c["kv_scale"] = 1.0, 1.0
    c["k"] = torch.zeros(c["k"].shape).to(dt)
    c["k"][c["table"][0, 7], :, 3, 0] = torch.tensor(10.0).to(dt)
    gen = torch.Generator().manual_seed(3)
    c["v"] = (torch.randn(c["v"].shape, generator=gen) + 1.0).to(dt)
    c["q"] = torch.zeros(c["q"].shape, dtype=torch.bfloat16)
    c["q"][..., 0] = 1.0
    c = gpu(c)
    got = call(c)
    out, bound = ref64.tree(c["q"], c["k"], c["v"], c["table"].cpu(), c["lens"].cpu(), c["indptr"].cpu(),
                            c["mask"].cpu(), 1.0)
    ref64.assert_attention(got, out, bound)


def test_padded_pools():
    """Strides other than the dense ones: heads and pages with room between them."""
    c = gpu(make([300, 90], [9, 4], 8, 2, 128, seed=14))
    nb = c["k"].shape[0]
    for n in ("k", "v"):
        wide = torch.full((nb, 3, PAGE, 136), math.nan, dtype=torch.bfloat16, device=DEV)
        wide[:, :2, :, :128] = c[n]
        c[n] = wide[:, :2, :, :128]
    check(c, call(c))


def test_bad_trees_and_pages_are_flagged_and_nothing_else_is_touched():
    c = gpu(make([60, 60, 60, 60], [4, 4, 4, 4], 8, 2, 128, seed=15))
    good = call(c)
    assert pa.device_status() == 0
    lens, indptr, table = c["lens"].clone(), c["indptr"].clone(), c["table"].clone()
    c["lens"][1] = 3                        # fewer tokens than nodes
    got = call(c)
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
    assert torch.equal(got[:4], good[:4]) and torch.equal(got[8:], good[8:]) and bool((got[4:8] == 7).all())
    c["lens"] = lens
    c["indptr"] = torch.tensor([0, 4, 8, 12, 99], dtype=torch.int32, device=DEV)   # rows past the end
    got = call(c)
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
    assert torch.equal(got[:12], good[:12]) and bool((got[12:] == 7).all())
    c["indptr"] = torch.tensor([0, 4, 2, 12, 16], dtype=torch.int32, device=DEV)   # not ascending
    got = call(c)
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
    assert torch.equal(got[12:], good[12:])
    c["indptr"] = indptr
    for bad in (-1, c["k"].shape[0], 2 ** 31 - 1):
        c["table"] = table.clone()
        c["table"][2, 1] = bad              # 16 tokens of sequence 2 take no part
        got = call(c)
        assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
        assert torch.equal(got[:8], good[:8]) and torch.equal(got[12:], good[12:])
        assert torch.isfinite(got).all()
    c["table"] = table
    c["lens"] = torch.tensor([60, 60, 60, 10 ** 6], dtype=torch.int32, device=DEV)
    got = call(c)
    assert pa.device_status() & 1 << pa.PA_ERR_DEVICE_BOUNDS
    assert torch.equal(got[:12], good[:12])


@pytest.mark.parametrize("fp8", [False, True])
def test_row_tiles_side_by_side_and_one_after_another(fp8):
    """Trees of several row tiles, all alike and of very different sizes, over keys that many CTAs
    share; a sequence without the other sequences' second row tile among them."""
    for nodes in ([64, 64, 64], [64, 40, 33], [64, 5, 60], [64, 3, 2], [200, 190, 5], [100, 1, 0]):
        c = gpu(make([3000, 1700, 900], nodes, 8, 2, 128, seed=sum(nodes), fp8=fp8))
        check(c, call(c), what=str(nodes))
    assert pa.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hd,nq,nkv,nodes", [(64, 3, 1, [3]), (128, 8, 2, [20]), (256, 2, 1, [5]), (128, 4, 1, [40])])
def test_one_long_sequence_in_many_pieces(hd, nq, nkv, nodes, fp8):
    c = gpu(make([9000 + nodes[0]], nodes, nq, nkv, hd, seed=60 + hd, fp8=fp8))
    got = call(c)
    check(c, got)
    assert torch.equal(got, call(c))
    assert pa.device_status() == 0


def test_empty_trees_and_sequences():
    c = gpu(make([40, 30, 50], [3, 0, 2], 4, 2, 128, seed=16))
    check(c, call(c))
    c = gpu(make([3, 0, 2], [3, 0, 2], 4, 2, 64, seed=17))
    check(c, call(c))
    assert pa.device_status() == 0


def test_results_do_not_depend_on_the_run_or_the_workspace():
    c = gpu(make([5000, 70, 3100], [16, 3, 9], 8, 2, 128, seed=18))
    first = call(c)
    ws = space(c, extra=4096)
    ws.fill_(255)                            # NaN everywhere: nothing in it is read unwritten
    for _ in range(3):
        assert torch.equal(call(c, ws=ws), first)


def test_two_streams_with_their_own_workspaces():
    a, b = (gpu(make([900, 300], [12, 5], 8, 2, 128, seed=s)) for s in (19, 20))
    want = [call(a), call(b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [space(a), space(b)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [torch.full_like(c["q"], 7.0) for c in (a, b)]
        torch.cuda.synchronize()
        for c, s, w, o in zip((a, b), streams, ws, got):
            call(c, out=o, ws=w, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_captured_call_replays_with_new_trees():
    c = gpu(make([700, 90, 333], [8, 3, 5], 8, 2, 128, seed=21, pad_rows=8))
    c["nodes"] = 16
    ws, out = space(c), torch.full_like(c["q"], 7.0)
    call(c, out=out, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, out=out, ws=ws)
    for seed, lens, nodes in ((22, [700, 90, 333], [2, 9, 5]), (23, [1, 20, 640], [1, 16, 7])):
        n = make(lens, nodes, 8, 2, 128, seed=seed, words=1)
        c["table"].fill_(2 ** 31 - 1)
        c["k"].fill_(math.nan), c["v"].fill_(math.nan)
        w, nb = n["table"].shape[1], n["k"].shape[0]
        c["table"][:, :w] = n["table"].to(DEV)
        c["k"][:nb], c["v"][:nb] = n["k"].to(DEV), n["v"].to(DEV)
        rows = n["q"].shape[0]
        c["q"][:rows], c["mask"][:rows] = n["q"].to(DEV), n["mask"].to(DEV)
        c["lens"].copy_(n["lens"]), c["indptr"].copy_(n["indptr"])
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(c, out, what=f"replay {seed}")


def test_a_long_cache_whose_offsets_pass_32_bits():
    """Pages at byte offsets beyond 2^32 of their pool."""
    nkv, hd = 8, 128
    nb = (1 << 32) // (nkv * PAGE * hd * 2) + 64         # 4.3 GB of bf16 per pool
    c = make([200, 90], [8, 5], 32, nkv, hd, seed=24)
    used = c["k"].shape[0]
    c = gpu(c)
    for n in ("k", "v"):
        big = torch.empty((nb, nkv, PAGE, hd), dtype=torch.bfloat16, device=DEV)
        big[nb - used:] = c[n]
        c["small_" + n], c[n] = c[n], big
    real = c["table"] < used
    c["table"] = torch.where(real, c["table"] + (nb - used), c["table"])
    got = call(c)
    c["table"] = torch.where(real, c["table"] - (nb - used), c["table"])
    c["k"], c["v"] = c.pop("small_k"), c.pop("small_v")
    check(c, got)


def test_many_sequences():
    """More sequences than one launch's lists hold."""
    n = 2500
    c = gpu(make([3 + i % 20 for i in range(n)], [1 + i % 3 for i in range(n)], 4, 2, 64, seed=25))
    check(c, call(c))
    assert pa.device_status() == 0


# ---- commit -------------------------------------------------------------------------------

def run_commit(c, pools, accepted, kept, **kw):
    new = torch.full((len(kept),), -5, dtype=torch.int32, device=DEV)
    pa.pa_tree_commit(pools[0::2], pools[1::2], c["table"], c["lens"], c["indptr"], accepted.to(DEV),
                      kept.to(DEV), new, c["nodes"], layout=c["layout"], **kw)
    return new


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_commit_moves_rows_bit_for_bit(hd, layout, fp8):
    c = gpu(make([40, 23, 100, 9, 31], [12, 23, 30, 9, 5], 4, 2, hd, seed=hd, fp8=fp8, layout=layout))
    pools = [c["k"].clone(), c["v"].clone(), c["v"].clone(), c["k"].clone(), c["k"].clone(), c["v"].clone()]
    accepted = torch.full((5, 23), -1, dtype=torch.int32)
    paths = [[0, 3, 4, 11], [], [1, 2, 5, 6, 7, 20, 21, 29], list(range(9)), [4]]
    for b, path in enumerate(paths):
        accepted[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
    kept = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    want, lens = ref64.commit(pools, c["table"].cpu(), c["lens"].cpu(), c["indptr"].cpu(), accepted, kept, layout)
    new = run_commit(c, pools, accepted, kept)
    for got, ref in zip(pools, want):
        assert torch.equal(got.cpu().view(torch.uint8), ref.view(torch.uint8))
    assert new.tolist() == lens
    assert pa.device_status() == 0


def test_commit_of_more_pools_than_a_launch_takes():
    c = gpu(make([40, 23], [12, 9], 4, 2, 64, seed=3))
    pools = [c["k"] + i for i in range(150)]
    accepted = torch.tensor([[2, 5, 8], [0, 8, 0]], dtype=torch.int32)
    kept = torch.tensor([3, 2], dtype=torch.int32)
    want, lens = ref64.commit(pools, c["table"].cpu(), c["lens"].cpu(), c["indptr"].cpu(), accepted, kept)
    new = run_commit(c, pools, accepted, kept)
    assert all(torch.equal(g.cpu().view(torch.uint8), w.view(torch.uint8)) for g, w in zip(pools, want))
    assert new.tolist() == lens


def test_commit_cuts_bad_paths_and_flags_them():
    c = gpu(make([40, 23, 30, 31], [12, 9, 4, 8], 4, 2, 64, seed=4))
    c["lens"][2] = 2                                      # fewer tokens than nodes
    accepted = torch.tensor([[2, 5, 5, 7], [3, 9, 10, 11], [0, 1, 2, 3], [-1, 2, 3, 4]], dtype=torch.int32)
    kept = torch.tensor([4, 2, 4, 9], dtype=torch.int32)
    pools = [c["k"].clone(), c["v"].clone()]
    want, lens = ref64.commit(pools, c["table"].cpu(), c["lens"].cpu(), c["indptr"].cpu(), accepted,
                              torch.tensor([4, 2, 0, 0]))
    new = run_commit(c, pools, accepted, kept)
    assert new.tolist() == [28 + 2, 14 + 1, 2, 23]
    assert all(torch.equal(g.cpu().view(torch.uint8), w.view(torch.uint8)) for g, w in zip(pools, want))
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
    c["lens"][2] = 30
    c["table"][0, 1] = c["k"].shape[0]
    run_commit(c, pools, accepted[:, :1].contiguous(), torch.tensor([1, 0, 0, 0]).int())
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS


def test_write_verify_commit_and_go_on():
    """Two speculative steps as a server runs them: drafted rows written, the tree verified, the
    accepted path committed, then a plain decode over the new length sees what a sequence
    that had been written token by token sees."""
    c = gpu(make([100, 50], [6, 6], 8, 2, 128, seed=31))
    k, v = c["k"].nan_to_num(0.0), c["v"].nan_to_num(0.0)
    C = c["lens"].cpu() - 6
    gen = torch.Generator().manual_seed(5)
    new_k, new_v = (torch.randn(12, 2, 128, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
    slots = torch.tensor([int(c["table"][b, (int(C[b]) + i) // PAGE]) * PAGE + (int(C[b]) + i) % PAGE
                          for b in range(2) for i in range(6)], dtype=torch.int64, device=DEV)
    pa.pa_write_cache(new_k, new_v, k, v, slots)
    c["k"], c["v"] = k, v
    check(c, call(c))
    path = torch.tensor([[0, 2, 5], [1, 3, 0]], dtype=torch.int32)
    kept = torch.tensor([3, 2], dtype=torch.int32)
    new = run_commit(c, [k, v], path, kept)
    straight_k, straight_v = k.clone(), v.clone()
    order = [0, 2, 5, 6 + 1, 6 + 3]
    where = torch.tensor([int(slots[j]) for j in (0, 1, 2, 6, 7)], dtype=torch.int64, device=DEV)
    pa.pa_write_cache(new_k[order], new_v[order], straight_k, straight_v, where)
    q = torch.randn(2, 8, 128, generator=gen).to(torch.bfloat16).to(DEV)
    got, want = torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode(got, q, k, v, c["table"], new, c["scale"])
    pa.pa_decode(want, q, straight_k, straight_v, c["table"], torch.tensor([97, 46], dtype=torch.int32, device=DEV), c["scale"])
    assert torch.equal(got, want)
    assert pa.device_status() == 0
