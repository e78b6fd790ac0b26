"""Timed cases of the rotary positions and of the beam search around the paged cache.

Four operators, each on real shapes of a serving step:

* ``rope``     q and k rotated to their positions (pa_rope);
* ``append``   q rotated, k rotated on its way into the paged cache, v put beside it
               (pa_rope_append);
* ``select``   the best continuations over the beams and the vocabulary of every request
               (pa_beam_select);
* ``reorder``  block tables and partial pages of every layer following the chosen beams
               (pa_beam_reorder).

With ``own`` false, ``run`` computes each in elementary torch operations; with ``own`` true
it makes the framework's calls.  Sizes and lengths come from the case alone, all values, page
ids and parents from the seed.
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
        # a decode step of a batch, q and k as slices of the fused projection
        dict(name="rope step", op="rope", tokens=64, q_heads=32, kv_heads=8, head_dim=128, rotary=128,
             interleaved=False, inverse=False, scaling="none", fused=True, far=4096),
        # prompts of long documents, frequencies scaled for them
        dict(name="rope prompts", op="rope", tokens=16384, q_heads=32, kv_heads=8, head_dim=128, rotary=128,
             interleaved=False, inverse=False, scaling="yarn", fused=True, far=131072),
        # the gradient's direction: half of a smaller head, neighbouring channels, an odd count
        dict(name="rope back partial", op="rope", tokens=5003, q_heads=24, kv_heads=8, head_dim=64, rotary=32,
             interleaved=True, inverse=True, scaling="none", fused=False, far=8192),
        # one short conversation on the smallest configuration: latency alone
        dict(name="append one", op="append", tokens=1, pad=0, q_heads=4, kv_heads=2, head_dim=64, rotary=64,
             interleaved=False, scaling="none", fused=True, far=100, fp8=False, layout="HND"),
        # a decode step padded to its captured batch, in an 8-bit cache
        dict(name="append step fp8", op="append", tokens=256, pad=19, q_heads=32, kv_heads=8, head_dim=128,
             rotary=128, interleaved=False, scaling="bands", fused=True, far=32768, fp8=True, layout="NHD"),
        # a prefill's chunk of many prompts
        dict(name="append prompts", op="append", tokens=16384, pad=0, q_heads=32, kv_heads=8, head_dim=128,
             rotary=128, interleaved=False, scaling="none", fused=True, far=8192, fp8=False, layout="HND"),
        # wide heads, a quarter rotated, 8-bit, an odd number of tokens
        dict(name="append d256 fp8", op="append", tokens=7001, pad=0, q_heads=16, kv_heads=8, head_dim=256,
             rotary=64, interleaved=True, scaling="linear", fused=False, far=65536, fp8=True, layout="HND"),
        # a single request, four beams
        dict(name="select one", op="select", requests=1, beams=4, vocab=32000, best=8, fp32=True, masked=0.0,
             finished=False),
        # an odd vocabulary, whose rows start at any 4 bytes; half of it ruled out by a grammar
        dict(name="select odd masked", op="select", requests=12, beams=5, vocab=50001, best=10, fp32=True,
             masked=0.5, finished=True),
        # a large batch of wide searches over a large vocabulary
        dict(name="select batch", op="select", requests=64, beams=8, vocab=128000, best=16, fp32=False,
             masked=0.0, finished=False),
        # the step after a single selection, one layer
        dict(name="reorder one", op="reorder", requests=1, beams=4, min_len=100, max_len=100, layers=1,
             q_heads=4, kv_heads=2, head_dim=64, fp8=False, layout="HND"),
        # all layers of a 32-layer model, 32 requests of four beams
        dict(name="reorder layers", op="reorder", requests=32, beams=4, min_len=70, max_len=400, layers=32,
             q_heads=32, kv_heads=8, head_dim=128, fp8=False, layout="HND"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "select", "select", "reorder"])
    kv_heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    head_dim = rng.choice([64, 128, 256])
    fp8, layout = rng.random() < 0.4, rng.choice(["HND", "NHD"])
    if op in ("rope", "append"):
        most = min(32768, (1 << 26) // ((group + 2) * kv_heads * head_dim))
        tokens = _between(rng, 1, most)
        case = dict(op=op, tokens=tokens, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim,
                    rotary=rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4, 2 * rng.randint(1, head_dim // 2)]),
                    interleaved=rng.random() < 0.4, scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                    fused=rng.random() < 0.5, far=_between(rng, 16, 1 << 20))
        if case["rotary"] == 2 and case["scaling"] == "ntk":
            case["scaling"] = "none"              # a single pair's base has no such scaling
        if op == "rope":
            case["inverse"] = rng.random() < 0.4
        else:
            case.update(pad=rng.choice([0, 0, rng.randint(0, tokens // 2)]), fp8=fp8, layout=layout)
        return case
    if op == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        vocab = _between(rng, 60, 260000)
        requests = _between(rng, 1, max(1, min(64, (1 << 25) // (beams * vocab))))
        return dict(op=op, requests=requests, beams=beams, vocab=vocab, best=rng.randint(1, min(2 * beams + 4, vocab)),
                    fp32=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.5, 0.99]),
                    finished=beams > 1 and rng.random() < 0.4)
    beams, layers = rng.choice([2, 3, 4, 5, 8, 13, 16]), _between(rng, 1, 16)
    requests = _between(rng, 1, 32)
    max_len = _between(rng, 16, max(40, min(4096, (1 << 26) // (requests * beams * kv_heads * head_dim * layers))))
    return dict(op=op, requests=requests, beams=beams, min_len=_between(rng, 1, max_len), max_len=max_len, layers=layers,
                q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, fp8=fp8, layout=layout)


# ---- sizes that the case alone gives ------------------------------------------------------

def _lens(case):
    """Length of each request's beams."""
    rng = random.Random(case["requests"] * 7919 + case["max_len"])
    lens = [_between(rng, case["min_len"], case["max_len"]) for _ in range(case["requests"])]
    lens[-1] = case["max_len"]
    return lens


def _parents(case):
    """The beam that each beam goes on from: a few of the best have most of the children; every
    fifth request or so has one slot that is left alone (-1), its hypothesis finished."""
    rng = random.Random(case["requests"] * 104729 + case["beams"])
    rows = []
    for _ in range(case["requests"]):
        row = [min(case["beams"] - 1, int(rng.expovariate(1.0) * case["beams"] / 2)) for _ in range(case["beams"])]
        if rng.random() < 0.2:
            row[rng.randrange(case["beams"])] = -1
        rows.append(row)
    return rows


def _dead(case):
    """[requests][beams]: 0 a live beam, 1 finished.  A request keeps a live beam."""
    rng = random.Random(case["requests"] * 31 + case["vocab"])
    return [[int(case["finished"] and b > 0 and rng.random() < 0.3) for b in range(case["beams"])]
            for _ in range(case["requests"])]


def work(case):
    nq, nkv, hd = (case.get(k, 0) for k in ("q_heads", "kv_heads", "head_dim"))
    elem = 1 if case.get("fp8") else 2
    if case["op"] == "rope":
        t = case["tokens"]
        return dict(bytes=t * (nq + nkv) * hd * 4 + t * 8, flops=3 * t * (nq + nkv) * case["rotary"])
    if case["op"] == "append":
        t = case["tokens"] - case["pad"]
        return dict(bytes=max(8, t * (nq * 4 + 2 * nkv * (2 + elem)) * hd + t * 16),
                    flops=3 * t * (nq + nkv) * case["rotary"])
    if case["op"] == "select":
        rows = sum(b == 0 for r in _dead(case) for b in r)
        return dict(bytes=rows * case["vocab"] * (4 if case["fp32"] else 2) +
                    case["requests"] * (case["beams"] * 4 + case["best"] * 12), flops=4 * rows * case["vocab"])
    moved = table = 0
    for n, row in zip(_lens(case), _parents(case)):
        away = sum(p >= 0 and p != j for j, p in enumerate(row))
        moved += away * (n % PAGE)
        table += away * (n // PAGE)
    return dict(bytes=max(4, moved * nkv * hd * elem * 2 * case["layers"] * 2 + table * 8), flops=0)


# ---- inputs -------------------------------------------------------------------------------

class State:
    pass


def _values(shape, gen, fp8=False):
    """N(0, 1) values, bf16 or E4M3 codes."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device="cuda")
    step = max(1, (1 << 27) // max(1, out[0].numel()))
    for s in range(0, shape[0], step):
        part = out[s:s + step]
        x = torch.randn(part.shape, generator=gen, device="cuda")
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
    globals()["_prepare_" + case["op"]](case, s, rng, gen)
    return s


SCALING = dict(none=dict(), linear=dict(factor=4.0), ntk=dict(factor=8.0),
               yarn=dict(factor=32.0, original_len=4096), bands=dict(factor=8.0, original_len=8192))
BASE = 10000.0


def _frequencies(case):
    """(angle per position of each pair, in 64 bits; factor on the rotated channels)."""
    n, kind = case["rotary"], case["scaling"]
    how = SCALING[kind]
    scale, length = how.get("factor", 1.0), how.get("original_len", 0)
    i = torch.arange(n // 2, dtype=torch.float64)
    f = BASE ** (-2 * i / n)
    if kind == "linear":
        return f / scale, 1.0
    if kind == "ntk":
        return (BASE * scale ** (n / (n - 2))) ** (-2 * i / n), 1.0
    if kind == "bands":            # long waves are slowed, short ones kept, a line between
        turns = length * f / (2 * math.pi)
        s = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f * ((1 - s) / scale + s), 1.0
    if kind == "yarn":
        def pair(turns):
            return n * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(BASE))
        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), n - 1)
        s = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (s / scale + 1 - s), 0.1 * math.log(scale) + 1
    return f, 1.0


def _prepare_rotation(case, s, rng, gen):
    t, nq, nkv, hd = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["fused"]:              # the slices of one projection's output
        x = _values((t, (nq + 2 * nkv) * hd), gen)
        s.q = x[:, :nq * hd].view(t, nq, hd)
        s.k = x[:, nq * hd:(nq + nkv) * hd].view(t, nkv, hd)
        s.v = x[:, (nq + nkv) * hd:].view(t, nkv, hd)
    else:
        s.q, s.k, s.v = (_values((t, h, hd), gen) for h in (nq, nkv, nkv))
    # a few sequences' runs of tokens, each from a position of its own
    pos, at = np.empty(t, np.int64), 0
    while at < t:
        n = min(t - at, int(rng.integers(1, 2 * (t // 8 + 1) + 1)))
        pos[at:at + n] = int(rng.integers(0, case["far"])) + np.arange(n)
        at += n
    s.pos = torch.from_numpy(pos).cuda()
    f, s.factor = _frequencies(case)
    s.freq = f.cuda()
    s.q_out = torch.zeros((t, nq, hd), dtype=torch.bfloat16, device="cuda")
    if own:
        import paged_kv_gqa_15_gb300 as pa
        s.turns, s.factor = pa.rope_table(case["rotary"], BASE, scaling=case["scaling"], **SCALING[case["scaling"]])


def _prepare_rope(case, s, rng, gen):
    _prepare_rotation(case, s, rng, gen)
    s.k_out = torch.zeros((case["tokens"], case["kv_heads"], case["head_dim"]), dtype=torch.bfloat16, device="cuda")


def _prepare_append(case, s, rng, gen):
    _prepare_rotation(case, s, rng, gen)
    t = case["tokens"]
    blocks = t // PAGE * 11 // 10 + 3
    s.slots = torch.from_numpy(rng.permutation(blocks * PAGE)[:t].astype(np.int64) if t <= 4096 else
                               # prompts: whole pages in a row
                               (rng.permutation(blocks)[:, None] * PAGE + np.arange(PAGE)).reshape(-1)[:t]).cuda()
    s.slots[t - case["pad"]:] = -1
    shape = _pool_shape(case, blocks)
    s.k_cache, s.v_cache = _values(shape, gen, case["fp8"]), _values(shape, gen, case["fp8"])
    s.scale = FP8_SCALE if case["fp8"] else 1.0


def _prepare_select(case, s, rng, gen):
    r, b, v = case["requests"], case["beams"], case["vocab"]
    x = torch.randn((r * b, v), generator=gen, device="cuda") * 2.0
    # a few tokens of every beam stand out, as after a sensible context
    few = torch.randint(v, (r * b, 12), generator=gen, device="cuda")
    x.scatter_add_(1, few, torch.rand((r * b, 12), generator=gen, device="cuda") * 8.0)
    if case["masked"]:
        out = torch.rand((r * b, v), generator=gen, device="cuda") < case["masked"]
        out[:, :40] = False        # what the grammar always allows
        x.masked_fill_(out, -math.inf)
    s.logits = x if case["fp32"] else x.to(torch.bfloat16)
    s.cum = -torch.rand((r, b), generator=gen, device="cuda") * 6.0 - 10.0
    if case["requests"] > 1 and b > 1:
        s.cum[0, 1:] = -math.inf   # a request at its first step: one beam alone is alive
    s.dead = torch.tensor(_dead(case), dtype=torch.uint8).cuda() if case["finished"] else None
    s.end = 2
    k = case["best"]
    s.scores = torch.empty((r, k), dtype=torch.float32, device="cuda")
    s.beams, s.tokens = (torch.empty((r, k), dtype=torch.int32, device="cuda") for _ in range(2))
    if own:
        import paged_kv_gqa_15_gb300 as pa
        s.space = pa.alloc_workspace(pa.beam_select_workspace_size(r, b, v), "cuda")


def _prepare_reorder(case, s, rng, gen):
    r, b = case["requests"], case["beams"]
    lens = np.repeat(np.array(_lens(case)), b)
    need = lens // PAGE + 1                                  # room for the next token
    blocks = int(need.sum())
    perm = rng.permutation(blocks)
    table = np.full((r * b, int(need.max())), -1, np.int32)
    for i, at in enumerate(np.cumsum(need) - need):
        table[i, :need[i]] = perm[at:at + need[i]]
    s.table = torch.from_numpy(table).cuda()
    s.lens = torch.from_numpy(lens.astype(np.int32)).cuda()
    s.parents = torch.tensor(_parents(case), dtype=torch.int32).cuda()
    shape = _pool_shape(case, blocks)
    s.pools = _values((2 * case["layers"] * shape[0],) + shape[1:], gen, case["fp8"]).view(
        (2 * case["layers"],) + shape)
    s.keys, s.vals = list(s.pools[0::2]), list(s.pools[1::2])


# ---- one pass -----------------------------------------------------------------------------

def run(s):
    return globals()["_run_" + s.case["op"]](s.case, s)


def _angles(s):
    """cos and sin [tokens][1][pairs]: the angles of far positions in 64 bits."""
    a = s.pos.double()[:, None] * s.freq
    return torch.cos(a).float()[:, None] * s.factor, torch.sin(a).float()[:, None] * s.factor


def _rotate(x, cos, sin, case):
    x, n = x.float(), case["rotary"]
    if case["interleaved"]:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
    else:
        a, b = x[..., :n // 2], x[..., n // 2:n]
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1 if case["interleaved"] else -2)
    return torch.cat([y.flatten(-2), x[..., n:]], -1)


def _run_rope(case, s):
    if own:
        import paged_kv_gqa_15_gb300 as pa
        pa.pa_rope(s.q_out, s.k_out, s.q, s.k, s.pos, s.turns, interleaved=case["interleaved"],
                   attention_factor=s.factor, inverse=case["inverse"])
        return s.q_out, s.k_out
    cos, sin = _angles(s)
    sin = -sin if case["inverse"] else sin
    return _rotate(s.q, cos, sin, case).to(torch.bfloat16), _rotate(s.k, cos, sin, case).to(torch.bfloat16)


def _run_append(case, s):
    if own:
        import paged_kv_gqa_15_gb300 as pa
        pa.pa_rope_append(s.q_out, s.q, s.k, s.v, s.k_cache, s.v_cache, s.slots, s.pos, s.turns,
                          layout=case["layout"], interleaved=case["interleaved"], attention_factor=s.factor,
                          k_scale=s.scale, v_scale=s.scale)
        return s.q_out, s.k_cache, s.v_cache
    real = s.slots >= 0
    cos, sin = _angles(s)
    q = _rotate(s.q, cos, sin, case).to(torch.bfloat16)
    q_out = torch.where(real[:, None, None], q, s.q_out)
    at = s.slots[real]
    for x, pool in ((_rotate(s.k, cos, sin, case), s.k_cache), (s.v.float(), s.v_cache)):
        x = x[real]
        if case["fp8"]:
            x = (x / s.scale).clamp(-448.0, 448.0)
        x = x.to(pool.dtype)
        pool, x = (pool.view(torch.uint8), x.view(torch.uint8)) if case["fp8"] else (pool, x)
        if case["layout"] == "HND":
            pool[at // PAGE, :, at % PAGE] = x
        else:
            pool[at // PAGE, at % PAGE] = x
    return q_out, s.k_cache, s.v_cache


def _run_select(case, s):
    r, b, v, k = case["requests"], case["beams"], case["vocab"], case["best"]
    if own:
        import paged_kv_gqa_15_gb300 as pa
        pa.pa_beam_select(s.scores, s.beams, s.tokens, s.logits, s.cum, s.space, finished=s.dead, end_token=s.end)
        return s.scores, s.beams, s.tokens
    # in 64 bits: candidates of two beams next to each other differ by less than 32 bits hold
    x = s.logits.view(r, b, v).double()
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    total = torch.exp(x - top).sum(-1, keepdim=True)
    score = s.cum.double()[..., None] + (x - (top + torch.log(total)))
    if s.dead is not None:
        gone = s.dead.bool()
        score = score.masked_fill(gone[..., None], -math.inf)
        score[..., s.end] = torch.where(gone, s.cum.double(), score[..., s.end])
    score = torch.where(torch.isnan(score), torch.full_like(score, -math.inf), score)
    best = torch.sort(score.view(r, b * v), dim=-1, descending=True, stable=True)
    value, at = best.values[:, :k], best.indices[:, :k]
    none = torch.isinf(value)
    beams, tokens = (at // v).masked_fill(none, -1), (at % v).masked_fill(none, -1)
    return value.float(), beams.to(torch.int32), tokens.to(torch.int32)


def _run_reorder(case, s):
    if own:
        import paged_kv_gqa_15_gb300 as pa
        pa.pa_beam_reorder(s.keys, s.vals, s.table, s.lens, s.parents, layout=case["layout"])
        return s.pools, s.table
    r, b = case["requests"], case["beams"]
    slot = torch.arange(r * b, device="cuda")
    parent = s.parents.flatten().long()
    parent = torch.where(parent >= 0, slot // b * b + parent, slot)
    full, rest = (s.lens // PAGE).long()[:, None], (s.lens % PAGE)[:, None]
    row = torch.arange(PAGE, device="cuda").expand(r * b, PAGE)
    to = torch.gather(s.table, 1, full).long().expand(r * b, PAGE)
    of = torch.where(row < rest, to[parent], to)             # rows past the length: onto themselves
    x = s.pools.view(torch.uint8) if case["fp8"] else s.pools
    if case["layout"] == "HND":
        x[:, to, :, row] = x[:, of, :, row]
    else:
        x[:, to, row] = x[:, of, row]
    col = torch.arange(s.table.shape[1], device="cuda")
    s.table = torch.where(col < full, s.table[parent], s.table)
    return s.pools, s.table


# ---- the definitions, in 64 bits ----------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, s)


def _exact_rotation(case, s, x, sign):
    """x turned pair by pair as complex numbers."""
    n, out = case["rotary"], x.double()
    angle = torch.remainder(sign * s.pos.double()[:, None] * s.freq, 2 * math.pi)
    turn = torch.polar(torch.full_like(angle, s.factor), angle)
    first = torch.arange(n // 2, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else n // 2)
    z = torch.complex(out[..., first], out[..., second]) * turn[:, None]
    out = out.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rope(case, s):
    sign = -1.0 if case["inverse"] else 1.0
    return _exact_rotation(case, s, s.q, sign), _exact_rotation(case, s, s.k, sign)


def _exact_append(case, s):
    n = case["tokens"] - case["pad"]
    q = s.q_out.double()
    q[:n] = _exact_rotation(case, s, s.q, 1.0)[:n]
    out = [q]
    for x, pool in ((_exact_rotation(case, s, s.k, 1.0), s.k_cache), (s.v.double(), s.v_cache)):
        got = pool.float().double()
        rows = got if case["layout"] == "NHD" else got.transpose(1, 2)       # [page][row][head][hd]
        x = (x[:n] / s.scale).clamp(-448.0, 448.0) if case["fp8"] else x[:n]
        rows[torch.div(s.slots[:n], PAGE, rounding_mode="floor"), s.slots[:n] % PAGE] = x
        out.append(got)
    return tuple(out)


def _exact_select(case, s):
    r, b, v, k = case["requests"], case["beams"], case["vocab"], case["best"]
    scores = torch.full((r, k), -math.inf, dtype=torch.float64)
    beams, tokens = torch.full((r, k), -1, dtype=torch.int32), torch.full((r, k), -1, dtype=torch.int32)
    for i in range(r):
        found = []
        for j in range(b):
            base = float(s.cum[i, j])
            if base == -math.inf:
                continue
            if s.dead is not None and int(s.dead[i, j]):
                found.append((-base, j, s.end))
                continue
            x = s.logits[i * b + j].double()
            x = base + torch.log_softmax(x, 0)
            floor = torch.topk(x, min(k, v)).values[-1]
            at = torch.nonzero((x >= floor) & ~torch.isinf(x))[:, 0]
            found += [(-y, j, t) for y, t in zip(x[at].tolist(), at.tolist())]
        for n, (y, j, t) in enumerate(sorted(found)[:k]):
            scores[i, n], beams[i, n], tokens[i, n] = -y, j, t
    return scores, beams, tokens


def _exact_reorder(case, s):
    before, old = s.pools.clone(), s.table.tolist()
    to, of = ((x.view(torch.uint8) if case["fp8"] else x) for x in (s.pools, before))
    new = [row[:] for row in old]
    for i, (n, row) in enumerate(zip(_lens(case), s.parents.tolist())):
        for j, p in enumerate(row):
            if p < 0 or p == j:
                continue
            a, c = i * case["beams"] + p, i * case["beams"] + j
            full, rest = divmod(n, PAGE)
            new[c][:full] = old[a][:full]
            src, dst = old[a][full], old[c][full]
            if case["layout"] == "HND":
                to[:, dst, :, :rest] = of[:, src, :, :rest]
            else:
                to[:, dst, :rest] = of[:, src, :rest]
    return s.pools, torch.tensor(new, dtype=torch.int32)
