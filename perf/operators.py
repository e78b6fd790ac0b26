"""Timed cases of the speculative and the sparse decode over the paged cache.

Four operators, each on real shapes of a serving step:

* ``tree``    attention of the drafted nodes of one token tree per sequence over that
              sequence's cache (pa_tree_decode);
* ``commit``  the K/V rows of the accepted path of every tree moved to the positions behind
              the context, in every layer's pools (pa_tree_commit);
* ``bounds``  per-page, per-channel minima and maxima of the keys (pa_page_bounds);
* ``sparse``  the pages that the bounds rank highest for this step's query, and the decode
              over those pages alone (pa_select_pages, pa_decode_pages).

With ``own`` false, ``run`` computes each in elementary torch operations; with ``own`` true
it makes the framework's calls.  Lengths come from the case alone, all values, page ids and
tree shapes from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
FP8_SCALE = 1.0 / 64          # N(0, 1) values over E4M3 codes up to 448 / 64 = 7


def listed():
    return [
        # one short conversation on the smallest configuration, an 8-node tree: latency alone
        dict(name="tree one short", op="tree", seqs=1, min_len=100, max_len=100, nodes=8, q_heads=4,
             kv_heads=2, head_dim=64, fp8=False, layout="HND", window=0),
        # a batch of 16 conversations verifying 16-node trees, the usual serving shape
        dict(name="tree batch", op="tree", seqs=16, min_len=512, max_len=4096, nodes=16, q_heads=32,
             kv_heads=8, head_dim=128, fp8=False, layout="HND", window=0),
        # long documents, few sequences: the key axis has to be split over the whole GPU
        dict(name="tree long", op="tree", seqs=8, min_len=32768, max_len=131072, nodes=24,
             q_heads=32, kv_heads=8, head_dim=128, fp8=False, layout="HND", window=0),
        # wide trees (256 query rows per kv head) over an 8-bit cache in the other page layout
        dict(name="tree wide fp8", op="tree", seqs=32, min_len=1000, max_len=8000, nodes=64,
             q_heads=32, kv_heads=8, head_dim=128, fp8=True, layout="NHD", window=0),
        # head_dim 256 with a sliding window, odd group and lengths
        dict(name="tree window d256", op="tree", seqs=24, min_len=700, max_len=9001, nodes=21,
             q_heads=24, kv_heads=8, head_dim=256, fp8=False, layout="HND", window=1024),
        # the step after a single verification, one layer
        dict(name="commit one", op="commit", seqs=1, min_len=100, max_len=100, nodes=8, q_heads=4,
             kv_heads=2, head_dim=64, fp8=False, layout="HND", layers=1),
        # all layers of a 32-layer model, 32 sequences
        dict(name="commit layers", op="commit", seqs=32, min_len=70, max_len=400, nodes=32,
             q_heads=32, kv_heads=8, head_dim=128, fp8=False, layout="HND", layers=32),
        # a decode step: each sequence's newest page
        dict(name="bounds step", op="bounds", seqs=64, min_len=512, max_len=4096, new=1, q_heads=32,
             kv_heads=8, head_dim=128, fp8=False, layout="HND"),
        # after a prefill: every page of long prompts
        dict(name="bounds prompts", op="bounds", seqs=8, min_len=8192, max_len=65536, new=0,
             q_heads=32, kv_heads=8, head_dim=128, fp8=False, layout="HND"),
        # the short end: one sequence of a few hundred pages
        dict(name="sparse one", op="sparse", seqs=1, min_len=6000, max_len=6000, q_heads=32,
             kv_heads=8, head_dim=128, fp8=False, layout="HND", pages=64, sink=1, recent=2),
        # long documents, 2048 tokens read of each
        dict(name="sparse long", op="sparse", seqs=8, min_len=32768, max_len=131072, q_heads=32,
             kv_heads=8, head_dim=128, fp8=False, layout="HND", pages=128, sink=1, recent=4),
        # a larger batch over an 8-bit cache, groups of 7, an odd page budget
        dict(name="sparse batch fp8", op="sparse", seqs=48, min_len=2000, max_len=33000, q_heads=28,
             kv_heads=4, head_dim=128, fp8=True, layout="NHD", pages=75, sink=2, recent=3),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "commit", "bounds", "sparse", "sparse"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    head_dim = rng.choice([64, 128, 256])
    case = dict(op=op, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim,
                fp8=rng.random() < 0.4, layout=rng.choice(["HND", "NHD"]))
    # tokens * kv heads * head_dim of a drawn cache: at most a quarter of the largest listed one
    room = 1 << 27
    seqs = _between(rng, 1, 64)
    top = max(40, min(65536, room // (seqs * kv_heads * head_dim)))
    max_len = _between(rng, 33, top)
    min_len = _between(rng, max(1, min(32, max_len)), max_len)
    case.update(seqs=seqs, min_len=min_len, max_len=max_len)
    if op == "tree":
        case.update(nodes=_between(rng, 1, min(min_len, 64, 256 // group)),
                    window=rng.choice([0, 0, 0, _between(rng, 16, 4096)]))
    elif op == "commit":
        layers = _between(rng, 1, 16)
        max_len = min(max_len, max(40, (room // 2) // (seqs * kv_heads * head_dim * layers)))
        case.update(max_len=max_len, min_len=min(min_len, max_len), layers=layers)
        case["nodes"] = _between(rng, 1, min(case["min_len"], 64))
    elif op == "bounds":
        case["new"] = rng.choice([0, 1, _between(rng, 2, max(2, min_len))])
    else:
        recent, sink = rng.randint(1, 5), rng.randint(0, 3)
        case.update(sink=sink, recent=recent, pages=sink + recent + _between(rng, 1, 256))
    return case


# ---- sizes that the case alone gives ------------------------------------------------------

def _lens(case):
    rng = random.Random(case["seqs"] * 7919 + case["max_len"])
    lens = [_between(rng, case["min_len"], case["max_len"]) for _ in range(case["seqs"])]
    lens[-1] = case["max_len"]
    return lens


def _nodes(case):
    """Drafted nodes per sequence: ragged, between half the largest tree and all of it."""
    rng = random.Random(case["nodes"] * 104729 + case["seqs"])
    n = [rng.randint((case["nodes"] + 1) // 2, case["nodes"]) for _ in range(case["seqs"])]
    n[0] = case["nodes"]
    return n


def _accepted_lens(case):
    """Accepted nodes per sequence: a few, as verification leaves them, sometimes none."""
    rng = random.Random(case["nodes"] * 31 + case["seqs"])
    return [min(n, rng.randint(0, 6)) if b else min(n, 4) for b, n in enumerate(_nodes(case))]


def _pages_of(n):
    return (n + PAGE - 1) // PAGE


def work(case):
    lens, nkv, nq, hd = _lens(case), case["kv_heads"], case["q_heads"], case["head_dim"]
    elem = 1 if case["fp8"] else 2
    if case["op"] == "tree":
        nodes, w = _nodes(case), case["window"]
        ctx = [n - t for n, t in zip(lens, nodes)]
        seen = [min(c, w) if w else c for c in ctx]
        keys = sum(c + t for c, t in zip(seen, nodes))
        rows = sum(nodes)
        return dict(bytes=keys * nkv * hd * 2 * elem + 2 * rows * nq * hd * 2 + rows * 8,
                    flops=4 * hd * nq * sum(t * (c + 1) for c, t in zip(seen, nodes)))
    if case["op"] == "commit":
        moved = sum(_accepted_lens(case))
        return dict(bytes=max(1, 2 * moved * nkv * hd * elem * 2 * case["layers"] + 16 * len(lens)),
                    flops=0)
    if case["op"] == "bounds":
        new = [min(n, case["new"]) if case["new"] else n for n in lens]
        rows = sum(n - (n - a) // PAGE * PAGE for n, a in zip(lens, new))
        pages = sum(_pages_of(n) - (n - a) // PAGE for n, a in zip(lens, new))
        return dict(bytes=(rows + 2 * pages) * nkv * hd * elem, flops=2 * rows * nkv * hd)
    pages = [_pages_of(n) for n in lens]
    kept = [min(p, case["pages"]) for p in pages]
    keys = sum(k * PAGE for k in kept)
    return dict(bytes=(sum(pages) * 2 + keys * 2) * nkv * hd * elem + 2 * len(lens) * nq * hd * 2,
                flops=4 * hd * nq * keys + 4 * hd * nkv * sum(pages))


# ---- inputs -------------------------------------------------------------------------------

class State:
    pass


def _values(shape, gen, fp8, drift=None):
    """N(0, 1) cache values, bf16 or E4M3 codes; drift: each page's keys share an offset, as
    neighbouring tokens' keys do."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device="cuda")
    step = max(1, (1 << 27) // max(1, out[0].numel()))
    for s in range(0, shape[0], step):
        part = out[s:s + step]
        x = torch.randn(part.shape, generator=gen, device="cuda")
        if drift is not None:
            x += drift(part.shape, gen)
        part.copy_(x.div_(FP8_SCALE).clamp_(-448.0, 448.0) if fp8 else x)
    return out


def _pool_shape(case, blocks):
    return ((blocks, case["kv_heads"], PAGE, case["head_dim"]) if case["layout"] == "HND" else
            (blocks, PAGE, case["kv_heads"], case["head_dim"]))


def prepare(case, seed):
    s = State()
    s.case = case
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens = np.array(_lens(case))
    need = (lens + PAGE - 1) // PAGE
    s.blocks = int(need.sum() * 11 // 10 + 1)
    perm = rng.permutation(s.blocks)
    table = np.full((len(lens), int(need.max())), np.iinfo(np.int32).max, np.int32)
    for b, at in enumerate(np.cumsum(need) - need):
        table[b, :need[b]] = perm[at:at + need[b]]
    s.table = torch.from_numpy(table).cuda()
    s.lens = torch.from_numpy(lens.astype(np.int32)).cuda()
    s.scale = 1.0 / math.sqrt(case["head_dim"])
    s.kv_scale = FP8_SCALE if case["fp8"] else 1.0
    s.max_len = int(lens.max())
    globals()["_prepare_" + case["op"]](case, s, rng, gen)
    return s


def _trees(case, rng):
    """Random parents (-1: child of the context), the tree masks as int64 words, and indptr."""
    nodes = _nodes(case)
    words = (case["nodes"] + 63) // 64
    mask = np.zeros((sum(nodes), words), np.uint64)
    at = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    for b, n in enumerate(nodes):
        seen = []
        for i in range(n):
            p = int(rng.integers(max(-1, i - 6), i)) if i else -1
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
            for w in range(words):
                mask[at[b] + i, w] = seen[i] >> 64 * w & 0xFFFFFFFFFFFFFFFF
    return at, mask.view(np.int64)


def _prepare_tree(case, s, rng, gen):
    at, mask = _trees(case, rng)
    s.indptr, s.mask = torch.from_numpy(at).cuda(), torch.from_numpy(mask).cuda()
    s.nodes = case["nodes"]
    shape = _pool_shape(case, s.blocks)
    s.k, s.v = _values(shape, gen, case["fp8"]), _values(shape, gen, case["fp8"])
    s.q = _values((int(at[-1]), case["q_heads"], case["head_dim"]), gen, False)
    s.out = torch.empty_like(s.q)
    s.space = None
    if own:
        import paged_kv_gqa_15_gb300 as pa
        s.space = pa.alloc_workspace(pa.tree_decode_workspace_size(
            case["seqs"], case["nodes"], case["q_heads"], case["kv_heads"], case["head_dim"]), "cuda")


def _prepare_commit(case, s, rng, gen):
    nodes, kept = _nodes(case), _accepted_lens(case)
    s.indptr = torch.from_numpy(np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)).cuda()
    s.nodes = case["nodes"]
    path = np.full((len(nodes), max(1, max(kept))), -1, np.int32)
    for b, (n, a) in enumerate(zip(nodes, kept)):
        path[b, :a] = np.sort(rng.choice(n, a, replace=False))
    s.path, s.kept = torch.from_numpy(path).cuda(), torch.tensor(kept, dtype=torch.int32).cuda()
    shape = _pool_shape(case, s.blocks)
    s.pools = _values((2 * case["layers"] * shape[0],) + shape[1:], gen, case["fp8"]).view(
        (2 * case["layers"],) + shape)
    s.keys, s.vals = list(s.pools[0::2]), list(s.pools[1::2])
    s.new_lens = torch.empty_like(s.lens)


def _prepare_bounds(case, s, rng, gen):
    s.k = _values(_pool_shape(case, s.blocks), gen, case["fp8"])
    s.first = torch.clamp(s.lens - case["new"], min=0) if case["new"] else None
    s.new = min(case["new"] or s.max_len, s.max_len)
    # one page more than the pool: the plain form's place for what it does not write
    s.room = torch.zeros((s.blocks + 1, case["kv_heads"], 2, case["head_dim"]), dtype=s.k.dtype,
                         device="cuda")
    s.bounds = s.room[:s.blocks]


def _page_drift(case):
    def drift(shape, gen):
        page = ((shape[0], shape[1], 1, shape[3]) if case["layout"] == "HND" else
                (shape[0], 1, shape[2], shape[3]))
        return torch.randn(page, generator=gen, device="cuda")
    return drift


def _prepare_sparse(case, s, rng, gen):
    shape = _pool_shape(case, s.blocks)
    s.k = _values(shape, gen, case["fp8"], _page_drift(case))
    s.v = _values(shape, gen, case["fp8"])
    s.q = _values((case["seqs"], case["q_heads"], case["head_dim"]), gen, False)
    rows = 2 if case["layout"] == "HND" else 1
    # the bounds that the program has kept so far: a newest page's rows past the sequence
    # take no part (each page belongs to one sequence)
    fill = torch.full((s.blocks,), PAGE, dtype=torch.int64, device="cuda")
    last = ((s.lens - 1) // PAGE).long()
    fill[s.table[torch.arange(case["seqs"], device="cuda"), last].long()] = s.lens.long() - last * PAGE
    keep = (torch.arange(PAGE, device="cuda") < fill[:, None])
    keep = keep[:, None, :, None] if rows == 2 else keep[:, :, None, None]
    s.bounds = torch.empty((s.blocks, case["kv_heads"], 2, case["head_dim"]), dtype=s.k.dtype,
                           device="cuda")
    step = max(1, (1 << 27) // max(1, s.k[0].numel()))
    for a in range(0, s.blocks, step):
        x, m = s.k[a:a + step].float(), keep[a:a + step]
        s.bounds[a:a + step, :, 0] = x.masked_fill(~m, math.inf).amin(rows).to(s.k.dtype)
        s.bounds[a:a + step, :, 1] = x.masked_fill(~m, -math.inf).amax(rows).to(s.k.dtype)
    s.out = torch.empty_like(s.q)
    s.pages = torch.empty((case["seqs"], case["kv_heads"], case["pages"]), dtype=torch.int32,
                          device="cuda")
    s.page_lens = torch.empty(case["seqs"], dtype=torch.int32, device="cuda")
    if own:
        import paged_kv_gqa_15_gb300 as pa
        s.select_space = pa.alloc_workspace(pa.select_pages_workspace_size(
            case["seqs"], case["kv_heads"], s.table.shape[1]), "cuda")
        s.space = pa.alloc_workspace(pa.decode_split_workspace_size(
            case["seqs"], case["q_heads"], case["head_dim"], case["pages"] * PAGE), "cuda")


# ---- one pass -----------------------------------------------------------------------------

def run(s):
    return globals()["_run_" + s.case["op"]](s.case, s)


def _rows(pool, table, case, scale):
    """Tokens of a block table as float32 [B][kv heads][tokens][head_dim]; entries out of range
    read some page, whose tokens the callers mask."""
    x = pool[table.clamp(0, pool.shape[0] - 1).long()].float()
    x = x.transpose(2, 3) if case["layout"] == "NHD" else x      # [B][pages][heads][16][hd]
    x = x.transpose(1, 2).flatten(2, 3)
    return x * scale if scale != 1.0 else x


def _attend(q, k, v, seen, scale):
    """softmax(scale q k) v over the keys that `seen` names; rows that see none are zeros."""
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = x.sum(-1, keepdim=True)
    return torch.matmul(x / torch.where(total > 0, total, torch.ones_like(total)), v)


def _run_tree(case, s):
    if own:
        import paged_kv_gqa_15_gb300 as pa
        pa.pa_tree_decode(s.out, s.q, s.k, s.v, s.table, s.lens, s.indptr, s.mask, s.scale, s.nodes,
                          s.space, layout=case["layout"], sliding_window=case["window"],
                          k_scale=s.kv_scale, v_scale=s.kv_scale)
        return s.out
    B, T, nkv, hd = case["seqs"], s.nodes, case["kv_heads"], case["head_dim"]
    total, g = s.q.shape[0], case["q_heads"] // case["kv_heads"]
    k, v = (_rows(p, s.table, case, s.kv_scale) for p in (s.k, s.v))
    count = s.indptr[1:] - s.indptr[:-1]
    node = torch.arange(T, device="cuda")
    real = node < count[:, None]                                   # [B][T]
    row = torch.where(real, s.indptr[:-1, None] + node, torch.full_like(s.indptr[:-1, None], total))
    rows = row.clamp(max=total - 1).long()
    q = s.q[rows].float().view(B, T, nkv, g, hd).permute(0, 2, 3, 1, 4).reshape(B, nkv, g * T, hd)
    bits = (s.mask[rows][..., None] >> torch.arange(64, device="cuda")) & 1     # [B][T][words][64]
    bits = bits.flatten(2).bool() & (torch.arange(bits.shape[2] * 64, device="cuda") < count[:, None, None])
    ctx = (s.lens - count)[:, None, None]                           # [B][1][1]
    key = torch.arange(k.shape[2], device="cuda")
    seen = (key < ctx).expand(B, T, -1)
    if case["window"]:
        seen = seen & (key >= ctx + bits.sum(-1, keepdim=True) - case["window"])
    at = key - ctx                                                  # drafted node of a key
    mine = torch.gather(bits, 2, at.clamp(0, bits.shape[2] - 1).expand(B, T, -1))
    seen = seen | (mine & (at >= 0) & (at < count[:, None, None]))
    o = _attend(q, k, v, seen.repeat(1, g, 1)[:, None], s.scale)
    o = o.view(B, nkv, g, T, hd).permute(0, 3, 1, 2, 4).reshape(B * T, case["q_heads"], hd)
    out = torch.empty((total + 1,) + tuple(s.q.shape[1:]), dtype=torch.bfloat16, device="cuda")
    out[row.flatten().long()] = o.to(torch.bfloat16)
    return out[:total]


def _place(s, pos):
    """(page, row) of token positions [B][n], which lie inside their sequences."""
    page = torch.gather(s.table, 1, (pos // PAGE).long()).long()
    return page, (pos % PAGE).long()


def _run_commit(case, s):
    if own:
        import paged_kv_gqa_15_gb300 as pa
        pa.pa_tree_commit(s.keys, s.vals, s.table, s.lens, s.indptr, s.path, s.kept, s.new_lens,
                          s.nodes, layout=case["layout"])
        return s.pools, s.new_lens
    ctx = (s.lens - (s.indptr[1:] - s.indptr[:-1]))[:, None]
    i = torch.arange(s.path.shape[1], device="cuda")
    to = torch.minimum(ctx + i, s.lens[:, None] - 1)     # past the path: a row onto itself
    src, dst = _place(s, torch.where(i < s.kept[:, None], ctx + s.path, to)), _place(s, to)
    x = s.pools.view(torch.uint8) if case["fp8"] else s.pools
    if case["layout"] == "HND":
        x[:, dst[0], :, dst[1]] = x[:, src[0], :, src[1]]
    else:
        x[:, dst[0], dst[1]] = x[:, src[0], src[1]]
    s.new_lens = ctx[:, 0] + s.kept
    return s.pools, s.new_lens


def _run_bounds(case, s):
    if own:
        import paged_kv_gqa_15_gb300 as pa
        pa.pa_page_bounds(s.bounds, s.k, s.table, s.lens, s.new, first_tokens=s.first,
                          layout=case["layout"])
        return s.bounds
    start = (s.first if s.first is not None else torch.zeros_like(s.lens))[:, None] // PAGE
    n = min(s.table.shape[1], _pages_of(s.new) + 1)
    page = start + torch.arange(n, device="cuda")
    real = page * PAGE < s.lens[:, None]
    ids = torch.gather(s.table, 1, page.clamp(max=s.table.shape[1] - 1).long())
    x = s.k[ids.clamp(0, s.blocks - 1).long()]
    x = (x.transpose(2, 3) if case["layout"] == "NHD" else x).float()         # [B][n][heads][16][hd]
    keep = (page[..., None] * PAGE + torch.arange(PAGE, device="cuda") < s.lens[:, None, None])
    keep = keep[:, :, None, :, None]
    low = x.masked_fill(~keep, math.inf).amin(3)
    high = x.masked_fill(~keep, -math.inf).amax(3)
    to = torch.where(real, ids, torch.full_like(ids, s.blocks)).flatten().long()
    both = torch.stack([low, high], 3).flatten(0, 1).to(s.k.dtype)
    room, both = (s.room.view(torch.uint8), both.view(torch.uint8)) if case["fp8"] else (s.room, both)
    room[to] = both
    return s.bounds


def _run_sparse(case, s):
    if own:
        import paged_kv_gqa_15_gb300 as pa
        pa.pa_select_pages(s.pages, s.page_lens, s.q, s.bounds, s.table, s.lens, s.select_space,
                           sink_pages=case["sink"], recent_pages=case["recent"])
        pa.pa_decode_pages(s.out, s.q, s.k, s.v, s.pages, s.page_lens, s.scale, s.space,
                           layout=case["layout"], k_scale=s.kv_scale, v_scale=s.kv_scale)
        return s.out, s.pages, s.page_lens
    B, nkv, hd, most = case["seqs"], case["kv_heads"], case["head_dim"], case["pages"]
    g, P = case["q_heads"] // nkv, s.table.shape[1]
    n = (s.lens + PAGE - 1) // PAGE                                  # [B]
    # the ranking in 64 bits: pages next to the border differ by less than 32 bits hold
    q = s.q.double().view(B, nkv, g, hd)
    near = s.bounds[s.table.clamp(0, s.blocks - 1).long()].double()  # [B][P][heads][2][hd]
    score = (near[:, :, :, 1] * q.clamp(min=0).sum(2)[:, None] +
             near[:, :, :, 0] * q.clamp(max=0).sum(2)[:, None]).sum(-1).transpose(1, 2)
    page = torch.arange(P, device="cuda")
    held = ((page < case["sink"]) | (page >= n[:, None] - case["recent"]))[:, None]
    score = score.masked_fill(held, math.inf).masked_fill((page >= n[:, None])[:, None], -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :most]
    kept = torch.clamp(n, max=most)
    rank = torch.arange(best.shape[-1], device="cuda")
    best = torch.where(rank < kept[:, None, None], best, torch.full_like(best, P)).sort(-1).values
    ids = torch.gather(s.table[:, None].expand(B, nkv, P), 2, best.clamp(max=P - 1))
    ids = torch.where(best < P, ids, torch.full_like(ids, -1))
    s.pages = torch.full((B, nkv, most), -1, dtype=torch.int32, device="cuda")
    s.pages[..., :ids.shape[-1]] = ids
    s.page_lens = torch.minimum(kept * PAGE, kept * PAGE + s.lens - n * PAGE).to(torch.int32)
    head = torch.arange(nkv, device="cuda")[:, None]
    pick = s.pages.clamp(min=0).long()
    k, v = ((p[pick, head[None]] if case["layout"] == "HND" else p[pick, :, head[None]]).float()
            .flatten(2, 3) * s.kv_scale for p in (s.k, s.v))         # [B][heads][pages * 16][hd]
    seen = torch.arange(most * PAGE, device="cuda") < s.page_lens[:, None, None, None]
    o = _attend(s.q.float().view(B, nkv, g, hd), k, v, seen, s.scale)
    return o.view(B, nkv * g, hd).to(torch.bfloat16), s.pages, s.page_lens


# ---- the definitions, in 64 bits ----------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, s)


def _token(pool, case, s, b, pos):
    """Rows [kv heads][n][head_dim] of sequence b's tokens at `pos`, in 64 bits."""
    page = s.table[b].long()[pos // PAGE]
    got = pool[page, :, pos % PAGE] if case["layout"] == "HND" else pool[page, pos % PAGE]
    return got.double().permute(1, 0, 2) * s.kv_scale


def _exact_tree(case, s):
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    at, lens, masks = s.indptr.tolist(), s.lens.tolist(), s.mask.cpu().numpy().view(np.uint64)
    g = case["q_heads"] // case["kv_heads"]
    for b in range(case["seqs"]):
        n = at[b + 1] - at[b]
        ctx = lens[b] - n
        pos = torch.arange(lens[b], device="cuda")
        k, v = _token(s.k, case, s, b, pos), _token(s.v, case, s, b, pos)
        see = np.zeros((n, lens[b]), bool)
        for i in range(n):
            chain = [j for j in range(n) if int(masks[at[b] + i, j // 64]) >> (j % 64) & 1]
            low = max(0, ctx + len(chain) - case["window"]) if case["window"] else 0
            see[i, low:ctx] = True
            see[i, [ctx + j for j in chain]] = True
        see = torch.from_numpy(see).cuda()
        for h in range(case["q_heads"]):
            x = s.q[at[b]:at[b + 1], h].double() @ k[h // g].T * s.scale
            p = torch.softmax(x.masked_fill(~see, -math.inf), -1)
            out[at[b]:at[b + 1], h] = torch.nan_to_num(p) @ v[h // g]
    return out


def _exact_commit(case, s):
    before = s.pools.clone()
    to = s.pools.view(torch.uint8) if case["fp8"] else s.pools
    of = before.view(torch.uint8) if case["fp8"] else before
    at, lens, kept, path = s.indptr.tolist(), s.lens.tolist(), s.kept.tolist(), s.path.tolist()
    table, new = s.table.tolist(), []
    for b in range(case["seqs"]):
        ctx = lens[b] - (at[b + 1] - at[b])
        for i in range(kept[b]):
            j = ctx + path[b][i]
            a, c = table[b][j // PAGE], table[b][(ctx + i) // PAGE]
            if case["layout"] == "HND":
                to[:, c, :, (ctx + i) % PAGE] = of[:, a, :, j % PAGE]
            else:
                to[:, c, (ctx + i) % PAGE] = of[:, a, j % PAGE]
        new.append(ctx + kept[b])
    return s.pools, torch.tensor(new, dtype=torch.int32)


def _exact_bounds(case, s):
    for b, n in enumerate(s.lens.tolist()):
        start = max(0, n - case["new"]) // PAGE if case["new"] else 0
        ids = s.table[b].long()
        for which, rows in ((ids[start:n // PAGE], PAGE), (ids[n // PAGE:_pages_of(n)], n % PAGE)):
            if len(which) == 0:
                continue
            x = s.k[which].double()
            x = (x if case["layout"] == "HND" else x.transpose(1, 2))[:, :, :rows]
            s.bounds[which] = torch.stack([x.amin(2), x.amax(2)], 2).to(s.k.dtype)
    return s.bounds


def _exact_sparse(case, s):
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    g, lens = case["q_heads"] // case["kv_heads"], s.lens.tolist()
    pages = torch.full((case["seqs"], case["kv_heads"], case["pages"]), -1, dtype=torch.int32)
    kept = []
    for b in range(case["seqs"]):
        n = _pages_of(lens[b])
        ids = s.table[b, :n].long()
        count = min(n, case["pages"])
        kept.append(count * PAGE - (n * PAGE - lens[b]))
        for h in range(case["kv_heads"]):
            q = s.q[b, h * g:(h + 1) * g].double()
            low, high = s.bounds[ids, h, 0].double(), s.bounds[ids, h, 1].double()
            score = torch.zeros(n, dtype=torch.float64, device="cuda")
            for i in range(g):
                score += torch.maximum(q[i] * low, q[i] * high).sum(-1)
            held = [p for p in range(n) if p < case["sink"] or p >= n - case["recent"]][-case["pages"]:]
            if count == n:
                chosen = list(range(n))
            else:
                value = score.tolist()
                free = sorted(set(range(n)) - set(held), key=lambda p: (-value[p], p))
                chosen = sorted(held + free[:count - len(held)])
            pick = torch.tensor(chosen, device="cuda")
            pages[b, h, :count] = ids[pick].int().cpu()
            pos = (pick[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
            pos = pos[pos < lens[b]]
            k, v = (_token(p, case, s, b, pos)[h] for p in (s.k, s.v))
            out[b, h * g:(h + 1) * g] = torch.softmax(q @ k.T * s.scale, -1) @ v
    return out, pages, torch.tensor(kept, dtype=torch.int32)
