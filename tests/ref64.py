"""Plain 64-bit forms of the tree attention, the path commit, the page bounds and the page
selection, on CPU tensors: loops over sequences and heads, straight from the definitions.

bf16 outputs of the attention are compared element by element.  With p the softmax weights
and A = sum_j p_j |v_j|, an implementation that rounds each weight to bf16 (half a step:
2^-8 of its value, on the weights and not on their sum) and its result to bf16 is off by at
most 2^-8 A + 2^-8 |out|; scores in fp32 (head_dim products and sums, then a product with
the scale: a relative error below (head_dim + 8) 2^-24 of sum_d |q_d k_d| scale, which is
under 64 for the tests' inputs) move each weight by a factor 1 +- 64 (264) 2^-24 = 1.0e-3 at
most, and the normalisation by as much again: 2.1e-3 A.  Where an 8-bit cache is multiplied on
the 8-bit tensor cores, q and p are carried as sums of E4M3 values; `extra` adds what that
path documents."""
import math

import numpy as np
import torch

PAGE = 16
BF16 = 2.0 ** -8      # half a step of bf16, relative


def page_rows(pool, layout):
    """Pool as [blocks][heads][16][hd] in 64 bits (values of E4M3 codes)."""
    x = pool.detach().cpu()
    if x.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn)
    x = x.float().double()
    return x if layout == "HND" else x.transpose(1, 2)


def tokens(pool, table, n, layout, scale=1.0):
    """Rows [heads][n][hd] of the first n tokens of one block-table row."""
    rows = page_rows(pool, layout)
    pos = torch.arange(n)
    page = table.cpu().long()[pos // PAGE]
    return rows[page, :, pos % PAGE].permute(1, 0, 2) * scale


def attend(q, k, v, see, scale):
    """(out, sum_j p_j |v_j|) of rows q over keys k where see; rows that see none are zero."""
    x = (q @ k.T * scale).masked_fill(~see, -math.inf)
    p = torch.nan_to_num(torch.softmax(x, -1)) * see
    v = torch.where(see.any(0)[:, None], v, torch.zeros_like(v))   # unseen rows may hold NaN
    return p @ v, p @ v.abs()


def mask_bits(mask_row, n):
    words = [int(w) & 0xFFFFFFFFFFFFFFFF for w in mask_row.tolist()]
    return [j for j in range(n) if words[j // 64] >> (j % 64) & 1]


def tree(q, k_cache, v_cache, tables, lens, indptr, mask, scale, layout="HND", window=0,
         k_scale=1.0, v_scale=1.0):
    """(out, A) [rows][nq][hd] in 64 bits; rows of no sequence are NaN."""
    q = q.detach().cpu().double()
    nq = q.shape[1]
    nkv = page_rows(k_cache[:1], layout).shape[1]
    g = nq // nkv
    out = torch.full(q.shape, math.nan, dtype=torch.float64)
    bound = out.clone()
    at = indptr.tolist()
    for b in range(len(at) - 1):
        T, L = at[b + 1] - at[b], int(lens[b])
        C = L - T
        k = tokens(k_cache, tables[b], L, layout, k_scale)
        v = tokens(v_cache, tables[b], L, layout, v_scale)
        see = torch.zeros(T, L, dtype=torch.bool)
        for i in range(T):
            nodes = mask_bits(mask[at[b] + i], T)
            low = max(0, C + len(nodes) - window) if window > 0 else 0
            see[i, low:C] = True
            for j in nodes:
                see[i, C + j] = True
        for h in range(nq):
            # rows one by one: a NaN key that one row does not see is seen by another
            for i in range(T):
                o, a = attend(q[at[b] + i:at[b] + i + 1, h], torch.where(
                    see[i][:, None], k[h // g], torch.zeros_like(k[h // g])), v[h // g], see[i:i + 1], scale)
                out[at[b] + i, h], bound[at[b] + i, h] = o[0], a[0]
    return out, bound


def assert_attention(got, out, bound, extra=0.0, what=""):
    """got (bf16) within the rounding bound of (out, A); see the module's docstring."""
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    room = BF16 * out.abs() + (BF16 + 2.1e-3 + extra) * bound + 1e-30
    off = (got - out).abs() / room
    assert off.max() <= 1.0, f"{what}: {off.max():.3f} of the bound at {np.unravel_index(int(off.argmax()), off.shape)}"


def commit(pools, tables, lens, indptr, accepted, accept_lens, layout="HND"):
    """New pools (copies) and lengths; paths are cut before a bad entry."""
    out = [p.detach().cpu().clone() for p in pools]
    view = [p.view(torch.uint8) for p in out]
    old = [p.clone() for p in view]
    new = []
    for b in range(len(lens)):
        T = int(indptr[b + 1]) - int(indptr[b])
        C, last, n = int(lens[b]) - T, -1, 0
        for a in accepted[b].tolist()[:int(accept_lens[b])]:
            if a <= last or a >= T:
                break
            for o, v in zip(old, view):
                (p0, r0), (p1, r1) = ((int(tables[b][j // PAGE]), j % PAGE) for j in (C + a, C + n))
                if layout == "HND":
                    v[p1, :, r1] = o[p0, :, r0]
                else:
                    v[p1, r1] = o[p0, r0]
            last, n = a, n + 1
        new.append(C + n)
    return out, new


def bounds(before, k_cache, tables, lens, first, layout="HND"):
    """The bounds tensor after rewriting the pages that hold a token >= first[b]."""
    out = page_rows(before, "HND").clone()                  # [blocks][heads][2][hd]
    rows = page_rows(k_cache, layout)
    for b, n in enumerate(lens.tolist()):
        for p in range((n + PAGE - 1) // PAGE):
            if n > int(first[b]) and (p + 1) * PAGE > int(first[b]):
                i = int(tables[b][p])
                x = rows[i, :, :min(PAGE, n - p * PAGE)]
                out[i, :, 0], out[i, :, 1] = x.amin(1), x.amax(1)
    return out


def select(q, bnd, tables, lens, most, sink, recent):
    """(page_tables, page_lens) by exact scores: rational arithmetic is not needed, sums of at
    most 2 * 256 * 16 products of bf16 values are compared in 64 bits."""
    q = q.detach().cpu().double()
    bnd = page_rows(bnd, "HND")
    B, nq, _ = q.shape
    nkv = bnd.shape[1]
    g = nq // nkv
    out = torch.full((B, nkv, most), -1, dtype=torch.int32)
    kept = []
    for b in range(B):
        n = (int(lens[b]) + PAGE - 1) // PAGE
        c = min(n, most)
        kept.append(c * PAGE - (n * PAGE - int(lens[b])))
        for kh in range(nkv):
            score = []
            for p in range(n):
                i = int(tables[b][p])
                if not 0 <= i < bnd.shape[0]:
                    score.append(-math.inf)
                    continue
                s = 0.0
                for h in range(g):
                    x = q[b, kh * g + h]
                    t = torch.maximum(x * bnd[i, kh, 0], x * bnd[i, kh, 1])
                    s += float(torch.where(x == 0, torch.zeros_like(t), t).sum())
                score.append(math.inf if math.isnan(s) else s)
            if n <= most:
                pick = range(n)
            else:
                held = [p for p in range(n) if p < sink or p >= n - recent]
                free = sorted(range(sink, n - recent), key=lambda p: (-score[p], p))
                pick = sorted(held + free[:most - len(held)])
            for j, p in enumerate(pick):
                out[b, kh, j] = int(tables[b][p])
    return out, torch.tensor(kept, dtype=torch.int32)


def decode_pages(q, k_cache, v_cache, page_tables, page_lens, scale, layout="HND", k_scale=1.0,
                 v_scale=1.0):
    """(out, A) of the decode over per-head page lists."""
    q = q.detach().cpu().double()
    B, nq, hd = q.shape
    nkv = page_tables.shape[1]
    g = nq // nkv
    out, bound = torch.zeros(B, nq, hd, dtype=torch.float64), torch.zeros(B, nq, hd, dtype=torch.float64)
    for b in range(B):
        n = int(page_lens[b])
        for h in range(nq if n else 0):
            k = tokens(k_cache, page_tables[b, h // g], n, layout, k_scale)[h // g]
            v = tokens(v_cache, page_tables[b, h // g], n, layout, v_scale)[h // g]
            o, a = attend(q[b, h:h + 1], k, v, torch.ones(1, n, dtype=torch.bool), scale)
            out[b, h], bound[b, h] = o[0], a[0]
    return out, bound
