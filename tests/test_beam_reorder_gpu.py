"""pa_beam_reorder against a plain copy of everything (tests/rope_beam_ref.py), bit for bit, and a whole
beam search over the paged cache."""
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa
from tests import rope_beam_ref as ref
from tests.gpu_util import MAX_ABS, MEAN_ABS

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()
    yield
    assert pa.device_status() == 0


def make(R, B, lens, nkv, hd, layers, fp8=False, layout="HND", seed=1, extra=0):
    """Pools of random bits, a table whose rows share nothing, lengths [R * B]."""
    rng = np.random.default_rng(seed)
    lens = np.repeat(np.asarray(lens), B).astype(np.int32)
    need = lens // 16 + 1
    blocks = int(need.sum()) + 2
    perm = rng.permutation(blocks)
    table = np.full((R * B, int(need.max()) + extra), np.iinfo(np.int32).max, np.int32)
    for i, at in enumerate(np.cumsum(need) - need):
        table[i, :need[i]] = perm[at:at + need[i]]
    shape = (blocks, nkv, 16, hd) if layout == "HND" else (blocks, 16, nkv, hd)
    bits = [rng.integers(0, 256 if fp8 else 65536, shape).astype(np.uint8 if fp8 else np.uint16) for _ in range(2 * layers)]
    pools = [torch.from_numpy(b).to(DEV) if fp8 else torch.from_numpy(b.view(np.int16)).to(DEV).view(torch.bfloat16)
             for b in bits]
    return bits, pools, table, lens, rng


def bits_of(pool):
    x = pool if pool.dtype == torch.uint8 else pool.view(torch.int16)
    return x.cpu().numpy().view(np.uint8 if pool.dtype == torch.uint8 else np.uint16)


def check(bits, pools, table, lens, parents, layout="HND", skipped=None):
    """skipped: parents with the moves that are refused taken out."""
    t = torch.from_numpy(table).to(DEV)
    pa.pa_beam_reorder(pools[0::2], pools[1::2], t, torch.from_numpy(lens).to(DEV),
                       torch.from_numpy(parents.astype(np.int32)).to(DEV), layout=layout)
    want, want_t = ref.reorder(bits, table, lens, parents if skipped is None else skipped, layout)
    assert np.array_equal(t.cpu().numpy(), want_t)
    for got, w in zip(pools, want):
        assert np.array_equal(bits_of(got), w)
    return want, want_t


@pytest.mark.parametrize("R,B,lens,nkv,hd,layers,fp8,layout", [
    (1, 4, [100], 2, 64, 1, False, "HND"), (3, 4, [1, 16, 33], 2, 128, 2, False, "HND"), (1, 1, [7], 1, 64, 1, False, "HND"),
    (2, 5, [0, 47], 3, 256, 1, False, "NHD"), (2, 8, [15, 31], 8, 128, 3, True, "HND"), (2, 13, [64, 65], 2, 64, 1, True, "NHD"),
    (1, 16, [200], 4, 128, 2, False, "NHD"), (2, 32, [5, 30], 1, 64, 1, True, "HND"), (4, 3, [900, 1, 17, 300], 1, 256, 1, False, "HND"),
    (1, 2, [29], 2, 64, 70, False, "HND"),           # 140 pools: two launches
    (1, 20, [5000], 1, 64, 1, True, "HND"),          # more table columns than threads
])
def test_moves(R, B, lens, nkv, hd, layers, fp8, layout):
    bits, pools, table, lens, rng = make(R, B, lens, nkv, hd, layers, fp8, layout, seed=R + B + hd)
    for parents in (rng.integers(0, B, (R, B)), np.tile(np.roll(np.arange(B), 1), (R, 1)), np.zeros((R, B), int),
                    rng.integers(-1, B, (R, B)), np.tile(np.arange(B), (R, 1)), np.full((R, B), -1)):
        bits, table = check(bits, pools, table, lens, parents, layout)


def test_pools_with_gaps_and_wider_tables():
    bits, _, table, lens, rng = make(2, 4, [21, 40], 3, 64, 1, seed=5, extra=3)
    wide = torch.zeros((bits[0].shape[0], 5, 16, 64), dtype=torch.bfloat16, device=DEV)
    both = [wide, wide.clone()]
    views = [w[:, 1:4] for w in both]
    for v, b in zip(views, bits):
        v.copy_(torch.from_numpy(b.view(np.int16)).to(DEV).view(torch.bfloat16))
    bits = [bits_of(v.contiguous()) for v in views]
    t = torch.from_numpy(table).to(DEV)
    parents = rng.integers(0, 4, (2, 4))
    pa.pa_beam_reorder(views[:1], views[1:], t, torch.from_numpy(lens).to(DEV), torch.from_numpy(parents.astype(np.int32)).to(DEV))
    want, want_t = ref.reorder(bits, table, lens, parents)
    assert np.array_equal(t.cpu().numpy(), want_t)
    for v, w, b in zip(views, want, both):
        assert np.array_equal(bits_of(v.contiguous()), w)
        assert (b[:, 0] == 0).all() and (b[:, 4] == 0).all()


def test_moves_that_cannot_be_made_are_flagged():
    B = 4
    base = np.array([[1, 0, 3, 2]])

    def run(change, keep, extra=0):
        bits, pools, table, lens, _ = make(1, B, [37], 2, 64, 1, seed=9, extra=extra)
        parents = base.copy()
        table, lens, parents = change(table, lens, parents)
        skipped = parents.copy()
        skipped[0, keep] = -1
        assert pa.device_status() == 0
        check(bits, pools, table, lens, parents, skipped=skipped)
        assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS

    def parent(j, p):
        def change(t, n, of):
            of[0, j] = p
            return t, n, of
        return change

    def entry(j, page):
        def change(t, n, of):
            t[j, 2] = t[1, 2] if page is None else page
            return t, n, of
        return change

    def length(j, n_new):
        def change(t, n, of):
            n[j] = n_new
            return t, n, of
        return change
    run(parent(2, 4), [2])
    run(parent(0, -2), [0])
    run(parent(3, 1 << 30), [3])
    run(entry(0, -1), [0, 1])                        # nothing to write into, nothing to take from
    run(entry(0, 1 << 20), [0, 1])
    run(entry(0, None), [0, 1])                      # two beams with one page for their next tokens
    run(length(2, 36), [2, 3])                       # another length than its parent's
    run(length(0, -5), [0, 1])
    run(length(0, 1 << 20), [0, 1])
    run(length(1, 2147483647), [0, 1])


def test_pages_of_a_beam_out_of_the_search_may_be_anothers():
    bits, pools, table, lens, _ = make(1, 4, [37], 2, 64, 1, seed=10)
    table[3] = table[0]                              # retired; its pages have gone to the first
    check(bits, pools, table, lens, np.array([[1, 2, 0, -1]]))
    assert pa.device_status() == 0


def test_shared_prompt_becomes_a_beam_each():
    """After one prefill: every beam's table names the prompt's pages and, for the page that its next
    token goes to, one of its own; parents 0 give each its copy of the rows there."""
    bits, pools, table, lens, _ = make(1, 4, [45], 2, 128, 2, seed=11)
    own = table[:, 2].copy()
    table[1:, :2] = 0x7fff0000                       # not there yet
    parents = np.zeros((1, 4), int)
    _, after = check(bits, pools, table, lens, parents)
    assert (after[:, :2] == after[0, :2]).all() and np.array_equal(after[:, 2], own)


def test_a_beam_search_step_by_step():
    """Steps of a search over a random model: append with rotation, split decode, selection, reordering,
    captured once and replayed.  Each step's attention is compared with that over the tokens of every
    beam's own history, each selection with the one in 64 bits on the same logits."""
    R, B, nq, nkv, hd, V, prompt, steps = 2, 4, 8, 2, 64, 1201, 29, 22
    g = torch.Generator().manual_seed(77)
    emb = torch.randn((V, (nq + 2 * nkv) * hd), generator=g).to(torch.bfloat16)
    head = torch.randn((nq * hd, V), generator=g) * 0.25
    turns, m = pa.rope_table(hd)
    f, _ = ref.frequencies(hd)
    S, pages = R * B, (prompt + steps) // 16 + 1
    kc = torch.zeros((S * pages + 1, nkv, 16, hd), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.arange(S * pages, dtype=torch.int32, device=DEV).view(S, pages)
    slot_pages = table.clone()                       # a sequence's own pages
    lens = torch.zeros(S, dtype=torch.int32, device=DEV)
    tokens, cum = torch.zeros((R, B), dtype=torch.int32, device=DEV), torch.zeros((R, B), device=DEV)
    parents = torch.zeros((R, B), dtype=torch.int32, device=DEV)
    scores = torch.zeros((R, B), device=DEV)
    space = pa.alloc_workspace(pa.beam_select_workspace_size(R, B, V), DEV)
    dec = pa.alloc_workspace(pa.decode_split_workspace_size(S, nq, hd, pages * 16), DEV)
    emb_d, head_d = emb.to(DEV), head.to(DEV)
    slots = torch.zeros(S, dtype=torch.int64, device=DEV)
    pos = torch.zeros(S, dtype=torch.int64, device=DEV)
    qo = torch.empty((S, nq, hd), dtype=torch.bfloat16, device=DEV)
    att, logits = torch.empty_like(qo), torch.empty((S, V), device=DEV)

    def append(x):
        n = x.shape[0]
        return x[:, :nq * hd].view(n, nq, hd), x[:, nq * hd:-nkv * hd].view(n, nkv, hd), x[:, -nkv * hd:].view(n, nkv, hd)

    # prompts: written once, into the first beam's pages
    history = np.random.default_rng(78).integers(0, V, (R, prompt)).repeat(B, 0)
    for r in range(R):
        q, k, v = append(emb_d[torch.from_numpy(history[r * B]).to(DEV)])
        at = torch.arange(prompt, device=DEV)
        pa.pa_rope_append(None, None, k, v, kc, vc, slot_pages[r * B, at // 16].long() * 16 + at % 16, at, turns)
    lens.fill_(prompt)
    pa.pa_beam_reorder([kc], [vc], table, lens, parents)
    cum[:, 1:] = -math.inf                           # all beams are the prompt: one is searched
    tokens.copy_(torch.from_numpy(history[:, -1].reshape(R, B).astype(np.int32)))

    def step():
        """From each sequence's newest token to the tokens, parents and cache of the next."""
        q, k, v = append(emb_d[tokens.view(-1).long()])
        pos.copy_(lens)
        slots.copy_(torch.gather(slot_pages, 1, (lens // 16).long()[:, None])[:, 0].long() * 16 + lens % 16)
        lens.add_(1)
        pa.pa_rope_append(qo, q, k, v, kc, vc, slots, pos, turns)
        pa.pa_decode_split(att, qo, kc, vc, table, lens, 1 / math.sqrt(hd), pages * 16, dec)
        torch.matmul(att.view(S, -1).float(), head_d, out=logits)
        pa.pa_beam_select(scores, parents, tokens, logits, cum, space)
        cum.copy_(scores)
        pa.pa_beam_reorder([kc], [vc], table, lens, parents)

    state = [tokens, cum, lens, kc, vc, table, parents]
    saved = [t.clone() for t in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                       # warm up
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip(state, saved):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    moved = 0
    for i in range(steps):
        fed = tokens.cpu().numpy().reshape(-1)
        cum_in = cum.cpu().numpy().astype(np.float64)
        history = np.concatenate([history, fed[:, None]], 1)
        graph.replay()
        torch.cuda.synchronize()
        # attention over each beam's own history
        n = history.shape[1]
        want = np.zeros((S, nq, hd))
        for s in range(S):
            x = emb[torch.from_numpy(history[s])].double().numpy()
            q = ref.rotate(x[:, :nq * hd].reshape(n, nq, hd), np.arange(n), f)[-1]
            k = ref.rotate(x[:, nq * hd:-nkv * hd].reshape(n, nkv, hd), np.arange(n), f)
            v = x[:, -nkv * hd:].reshape(n, nkv, hd)
            for h in range(nq):
                w = k[:, h // (nq // nkv)] @ q[h] / math.sqrt(hd)
                w = np.exp(w - w.max())
                want[s, h] = w @ v[:, h // (nq // nkv)] / w.sum()
        err = np.abs(att.float().cpu().numpy() - want)
        assert err.max() <= MAX_ABS and err.mean() <= MEAN_ABS, (i, err.max(), err.mean())
        sc, bm, tk, closest = ref.select(logits.double().cpu().numpy(), cum_in, B)
        assert closest > 2.0 ** -19
        assert np.array_equal(parents.cpu().numpy(), bm) and np.array_equal(tokens.cpu().numpy(), tk)
        moved += int((bm != np.arange(B)).sum())
        history = history.reshape(R, B, n)[np.arange(R)[:, None], bm].reshape(S, n)
    assert moved > 20 and pa.device_status() == 0
