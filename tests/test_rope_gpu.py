"""pa_rope and pa_rope_append against the rotation in 64 bits (tests/rope_beam_ref.py)."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa
from tests import rope_beam_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()
    yield
    assert pa.device_status() == 0


def values(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def f64(t):
    return t.detach().float().cpu().double().numpy()


def check_rows(got, x, positions, f, m, interleaved, inverse=False, what=""):
    """A result is the exact one, off by what fp32 loses and half a step of bf16."""
    want = ref.rotate(f64(x), positions, f, interleaved, m, inverse)
    room = ref.rotation_slack(f64(x), len(f), interleaved, m)
    room = room + (np.abs(want) + room) * torch.finfo(torch.bfloat16).eps / 2
    err = np.abs(f64(got) - want)
    assert (err <= room).all(), f"{what}: off by {(err / np.maximum(room, 1e-30)).max():.3g} of what it may"
    n = 2 * len(f)
    assert torch.equal(got[..., n:].cpu().view(torch.int16), x[..., n:].cpu().view(torch.int16)), what


def some_positions(t, seed, far=40000):
    return np.random.default_rng(seed).integers(0, far, t)


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="bands", factor=8.0, original_len=8192),
            dict(scaling="yarn", factor=32.0, original_len=4096)]


@pytest.mark.parametrize("tokens,nq,nk,hd,rotary,interleaved", [
    (1, 4, 2, 64, 64, False), (1, 1, 1, 64, 2, True), (3, 32, 8, 128, 128, False), (7, 5, 3, 128, 128, True),
    (33, 16, 8, 256, 256, False), (2, 64, 8, 128, 64, False), (5, 24, 8, 256, 64, True), (4, 7, 1, 64, 16, False),
    (6, 3, 3, 64, 20, False), (6, 3, 3, 64, 20, True), (5, 2, 1, 128, 6, False), (5, 2, 1, 128, 126, True),
    (9, 1, 1, 256, 254, False), (257, 2, 2, 64, 32, False), (3, 96, 8, 256, 256, False),
    (2, 130, 1, 128, 128, True), (1000, 8, 1, 128, 128, False), (7000, 1, 1, 64, 64, True), (2500, 33, 7, 128, 128, False),
    (1500, 5, 2, 256, 100, False),
])
def test_rows(tokens, nq, nk, hd, rotary, interleaved):
    scaling = SCALINGS[(tokens + nq + rotary) % len(SCALINGS)]
    if rotary == 2:
        scaling = {}
    turns, m = pa.rope_table(rotary, **scaling)
    f, want_m = ref.frequencies(rotary, **scaling)
    assert m == pytest.approx(want_m, rel=2 ** -23)
    q, k = values((tokens, nq, hd), 1).to(DEV), values((tokens, nk, hd), 2).to(DEV)
    pos = some_positions(tokens, 3)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    for inverse in (False, True):
        pa.pa_rope(qo, ko, q, k, torch.from_numpy(pos).to(DEV), turns, interleaved=interleaved, attention_factor=m,
                   inverse=inverse)
        check_rows(qo, q, pos, f, want_m, interleaved, inverse, "q")
        check_rows(ko, k, pos, f, want_m, interleaved, inverse, "k")


@pytest.mark.parametrize("interleaved,rotary", [(False, 128), (True, 128), (False, 36)])
def test_far_and_negative_positions(interleaved, rotary):
    pos = np.array([0, 1, -1, 131071, 1 << 20, (1 << 20) + 1, (1 << 31) - 1, 1 << 31, -(1 << 31), 123456789])
    q = values((len(pos), 3, 128), 5).to(DEV)
    turns, _ = pa.rope_table(rotary, 500000.0)
    f, _ = ref.frequencies(rotary, 500000.0)
    out = torch.empty_like(q)
    pa.pa_rope(out, None, q, None, torch.from_numpy(pos).to(DEV), turns, interleaved=interleaved)
    # the fp64 angles are themselves off by 2^-53 of 2^31 turns' worth of radians, 2^-21 at most
    near = np.abs(pos) <= 1 << 20
    check_rows(out[torch.from_numpy(near).to(DEV)], q[torch.from_numpy(near).to(DEV)], pos[near], f, 1.0, interleaved)
    want = ref.rotate(f64(q), pos, f, interleaved)
    room = ref.rotation_slack(f64(q), len(f), interleaved) * 4
    assert (np.abs(f64(out) - want) <= room + (np.abs(want) + room) * 2.0 ** -8).all()
    # position 0 passes every channel
    assert torch.equal(out[0], q[0])


def test_frequencies_of_ones_own():
    f = np.array([1.0, 0.25, -0.5, 7.0, 0.0, 2 * np.pi])
    q = values((11, 2, 64), 8).to(DEV)
    pos = some_positions(11, 9, 5000)
    out = torch.empty_like(q)
    pa.pa_rope(out, None, q, None, torch.from_numpy(pos).to(DEV), pa.rope_table_of(f), interleaved=True,
               attention_factor=0.5)
    check_rows(out, q, pos, f, 0.5, True)


@pytest.mark.parametrize("interleaved,rotary", [(False, 128), (True, 128), (False, 44), (True, 64)])
def test_in_place_and_slices_of_a_projection(interleaved, rotary):
    t, nq, nk, hd = 37, 6, 2, 128
    x = values((t, (nq + 2 * nk) * hd), 11).to(DEV)
    turns, _ = pa.rope_table(rotary)
    f, _ = ref.frequencies(rotary)
    pos = some_positions(t, 12)
    at = torch.from_numpy(pos).to(DEV)
    cut = [nq * hd, (nq + nk) * hd]
    before = x.clone()
    q, k = x[:, :cut[0]].view(t, nq, hd), x[:, cut[0]:cut[1]].view(t, nk, hd)
    pa.pa_rope(q, k, q, k, at, turns, interleaved=interleaved)
    check_rows(q, before[:, :cut[0]].view(t, nq, hd), pos, f, 1.0, interleaved)
    check_rows(k, before[:, cut[0]:cut[1]].view(t, nk, hd), pos, f, 1.0, interleaved)
    assert torch.equal(x[:, cut[1]:], before[:, cut[1]:])          # the values beside them
    # heads first, as a transposed tensor has them, into a dense one
    y = values((nq, t, hd), 13).to(DEV)
    out = torch.empty((t, nq, hd), dtype=torch.bfloat16, device=DEV)
    pa.pa_rope(out, None, y.transpose(0, 1), None, at, turns, interleaved=interleaved)
    check_rows(out, y.transpose(0, 1), pos, f, 1.0, interleaved)
    back = torch.empty_like(y)
    pa.pa_rope(back.transpose(0, 1), None, y.transpose(0, 1), None, at, turns, interleaved=interleaved)
    assert torch.equal(back.transpose(0, 1), out)
    # one row for all tokens (an expanded input)
    one = values((1, nq, hd), 14).to(DEV).expand(t, nq, hd)
    pa.pa_rope(out, None, one, None, at, turns, interleaved=interleaved)
    check_rows(out, one, pos, f, 1.0, interleaved)


@pytest.mark.parametrize("interleaved,rotary", [(False, 64), (True, 20), (False, 12)])
def test_inverse_is_the_gradient(interleaved, rotary):
    """d/dx of sum(g * rotate(x)) by the formula's transposed map, and by differences of the 64-bit
    rotation (linear in x, so that a difference of any width is exact but for rounding)."""
    t, h, hd = 5, 2, 64
    turns, m = pa.rope_table(rotary, scaling="yarn", factor=8.0, original_len=512)
    f, want_m = ref.frequencies(rotary, scaling="yarn", factor=8.0, original_len=512)
    pos = some_positions(t, 21, 4096)
    g = values((t, h, hd), 22)
    dx = torch.empty_like(g, device=DEV)
    pa.pa_rope(dx, None, g.to(DEV), None, torch.from_numpy(pos).to(DEV), turns, interleaved=interleaved,
               attention_factor=m, inverse=True)
    check_rows(dx, g.to(DEV), pos, f, want_m, interleaved, True)
    x, dw = f64(values((t, h, hd), 23)), f64(g)
    slack = ref.rotation_slack(dw, len(f), interleaved, want_m)
    for c in range(0, hd, 3):
        up, down = x.copy(), x.copy()
        up[..., c] += 0.5
        down[..., c] -= 0.5
        slope = ((ref.rotate(up, pos, f, interleaved, want_m) - ref.rotate(down, pos, f, interleaved, want_m)) * dw).sum(-1)
        room = slack[..., c] + (np.abs(slope) + slack[..., c]) * 2.0 ** -8 + 1e-12
        assert (np.abs(f64(dx)[..., c] - slope) <= room).all()


def pools(blocks, nkv, hd, fp8, layout, seed):
    shape = (blocks, nkv, 16, hd) if layout == "HND" else (blocks, 16, nkv, hd)
    k, v = values(shape, seed, 60.0 if fp8 else 1.0), values(shape, seed + 1, 60.0 if fp8 else 1.0)
    return [(x.float().clamp(-448, 448).to(E4M3) if fp8 else x).to(DEV) for x in (k, v)]


def rows_of(pool, slots, layout):
    page, row = torch.div(slots, 16, rounding_mode="floor"), slots % 16
    x = pool.float()
    return x[page, :, row] if layout == "HND" else x[page, row]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens,nq,nkv,hd,rotary,interleaved,layout", [
    (1, 4, 2, 64, 64, False, "HND"), (1, 0, 1, 256, 256, True, "NHD"), (40, 32, 8, 128, 128, False, "HND"),
    (23, 7, 1, 128, 32, False, "NHD"), (23, 7, 1, 128, 34, False, "HND"), (17, 16, 8, 256, 64, True, "HND"),
    (300, 3, 3, 64, 10, True, "NHD"), (5, 64, 16, 128, 128, False, "HND"), (9, 2, 2, 256, 250, False, "NHD"),
    # more tokens than CTAs at a time
    (9001, 2, 1, 64, 64, False, "HND"), (4003, 20, 4, 128, 128, False, "NHD"), (3001, 16, 8, 256, 64, True, "HND"),
    (2999, 8, 2, 128, 38, True, "HND"),
])
def test_append(tokens, nq, nkv, hd, rotary, interleaved, layout, fp8):
    blocks = tokens // 16 + 3
    kc, vc = pools(blocks, nkv, hd, fp8, layout, 31)
    turns, m = pa.rope_table(rotary, scaling="yarn" if rotary > 16 else "none", factor=4.0, original_len=1024)
    f, want_m = ref.frequencies(rotary, scaling="yarn" if rotary > 16 else "none", factor=4.0, original_len=1024)
    x = values((tokens, (nq + 2 * nkv) * hd), 33).to(DEV)
    q = x[:, :nq * hd].view(tokens, nq, hd)
    k = x[:, nq * hd:(nq + nkv) * hd].view(tokens, nkv, hd)
    v = x[:, (nq + nkv) * hd:].view(tokens, nkv, hd)
    rng = np.random.default_rng(34)
    pos = some_positions(tokens, 35)
    slots = rng.permutation(blocks * 16)[:tokens]
    skip = rng.random(tokens) < 0.2 if tokens > 1 else np.zeros(tokens, bool)
    given = torch.from_numpy(np.where(skip, -1 - rng.integers(0, 3, tokens), slots)).to(DEV)
    ks, vs = ((1 / 64, 1 / 50) if tokens % 2 else (0.0137, 1 / 32)) if fp8 else (1.0, 1.0)
    q_out = torch.full((tokens, nq, hd), 3.0, dtype=torch.bfloat16, device=DEV)
    before = kc.clone(), vc.clone()
    pa.pa_rope_append(q_out if nq else None, q if nq else None, k, v, kc, vc, given, torch.from_numpy(pos).to(DEV), turns,
                      layout=layout, interleaved=interleaved, attention_factor=m, k_scale=ks, v_scale=vs)
    keep = torch.from_numpy(~skip).to(DEV)
    if nq:
        check_rows(q_out[keep], q[keep], pos[~skip], f, want_m, interleaved, what="q")
        assert (q_out[~keep] == 3.0).all()
    at = torch.from_numpy(slots).to(DEV)[keep]
    # the values: what the plain cache write puts there; everything else stays
    want_k, want_v = before[0].clone(), before[1].clone()
    pa.pa_write_cache(k.contiguous(), v.contiguous(), want_k, want_v, given, layout=layout, k_scale=ks, v_scale=vs)
    assert torch.equal(vc.view(torch.uint8), want_v.view(torch.uint8))
    got = rows_of(kc, at, layout)
    if fp8:
        want = ref.rotate(f64(k)[~skip], pos[~skip], f, interleaved, want_m) / ks
        room = ref.rotation_slack(f64(k)[~skip], len(f), interleaved, want_m) / ks + np.abs(want) * 2.0 ** -23
        # half a step of E4M3: 2^-4 of the value, 2^-10 below 2^-6
        room = room + np.maximum((np.abs(want) + room) * torch.finfo(E4M3).eps / 2, 2.0 ** -10)
        assert (np.abs(f64(got) - np.clip(want, -448, 448)) <= room).all()
    else:
        check_rows(got.to(torch.bfloat16), k[keep], pos[~skip], f, want_m, interleaved, what="k")
    left = torch.ones(blocks * 16, dtype=torch.bool, device=DEV)
    left[at] = False
    left = torch.nonzero(left)[:, 0]
    assert torch.equal(rows_of(kc, left, layout), rows_of(before[0], left, layout))


def test_append_at_position_zero_is_the_cache_write():
    for fp8 in (False, True):
        kc, vc = pools(4, 2, 128, fp8, "HND", 41)
        kw, vw = kc.clone(), vc.clone()
        k, v, q = (values((20, h, 128), s).to(DEV) for h, s in ((2, 42), (2, 43), (4, 44)))
        slots = torch.randperm(64, generator=torch.Generator().manual_seed(1))[:20].to(DEV)
        turns, _ = pa.rope_table(128)
        q_out = torch.empty_like(q)
        pa.pa_rope_append(q_out, q, k, v, kc, vc, slots, torch.zeros(20, dtype=torch.int64, device=DEV), turns,
                          k_scale=1 / 64, v_scale=1 / 64)
        pa.pa_write_cache(k, v, kw, vw, slots, k_scale=1 / 64, v_scale=1 / 64)
        assert torch.equal(kc.view(torch.uint8), kw.view(torch.uint8))
        assert torch.equal(vc.view(torch.uint8), vw.view(torch.uint8)) and torch.equal(q_out, q)


@pytest.mark.parametrize("scale", [0.0123, 0.1, 1 / 3, 3.0, 2.0 ** -9, 7e-5, 1.0, 447.0, 1e-38, 3e38, 2.0 ** -120])
def test_codes_are_those_of_the_division(scale):
    """Every bf16 value, at position 0: the codes of the cache write, which divides; borders between
    codes and quotients next to them among them."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).to(DEV)
    x = bits.view(512, 2, 64).contiguous()
    finite = torch.isfinite(x.float())
    turns, _ = pa.rope_table(64)
    for interleaved, table in ((False, turns), (True, turns), (False, pa.rope_table(6)[0])):
        kc, vc, kw, vw = (torch.zeros((32, 2, 16, 64), dtype=torch.uint8, device=DEV) for _ in range(4))
        y = torch.where(finite, x, torch.zeros_like(x))      # a pair of infinity and 0 turns to NaN
        slots = torch.arange(512, device=DEV)
        pa.pa_rope_append(None, None, y, x, kc, vc, slots, torch.zeros_like(slots), table, interleaved=interleaved,
                          k_scale=scale, v_scale=scale)
        pa.pa_write_cache(y, x, kw, vw, slots, k_scale=scale, v_scale=scale)
        differ = kc != kw                                    # -0 turned is +0 where its partner is not negative
        assert ((kc | kw)[differ] == 0x80).all()
        assert torch.equal(vc, vw)


def test_slots_outside_the_pool_are_flagged():
    kc, vc = pools(3, 2, 64, False, "HND", 51)
    before = kc.clone(), vc.clone()
    k, v, q = (values((4, 2, 64), s).to(DEV) for s in (52, 53, 54))
    q_out = torch.full_like(q, 2.0)
    turns, _ = pa.rope_table(64)
    slots = torch.tensor([48, 1 << 40, -7, 47], device=DEV)
    assert pa.device_status() == 0
    pa.pa_rope_append(q_out, q, k, v, kc, vc, slots, torch.arange(4, device=DEV), turns)
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
    assert (q_out[:3] == 2.0).all() and not (q_out[3] == 2.0).all()
    assert torch.equal(vc[2, :, 15], v[3])
    kc[2, :, 15], vc[2, :, 15] = before[0][2, :, 15], before[1][2, :, 15]
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])


def test_nothing_to_do_and_infinities():
    turns, _ = pa.rope_table(32)
    empty = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    pa.pa_rope(empty, None, empty, None, none, turns)
    kc, vc = pools(2, 4, 64, False, "HND", 61)
    pa.pa_rope_append(None, None, empty, empty, kc, vc, none, none, turns)
    # infinities and NaN stay in their own pairs
    q = values((2, 1, 64), 62).to(DEV)
    q[0, 0, 5], q[1, 0, 40] = float("inf"), float("nan")
    out = torch.empty_like(q)
    for interleaved in (False, True):
        pa.pa_rope(out, None, q, None, torch.tensor([3, 4], device=DEV), turns, interleaved=interleaved)
        pair = {5, 4} if interleaved else {5, 21}
        assert set(torch.nonzero(~torch.isfinite(out[0, 0]))[:, 0].tolist()) == pair
        assert torch.nonzero(~torch.isfinite(out[1, 0]))[:, 0].tolist() == [40]


def test_side_stream_and_graph():
    q, k = values((70, 8, 128), 71).to(DEV), values((70, 2, 128), 72).to(DEV)
    turns, _ = pa.rope_table(128)
    pos = torch.arange(70, device=DEV) + 1000
    want_q, want_k = torch.empty_like(q), torch.empty_like(k)
    pa.pa_rope(want_q, want_k, q, k, pos, turns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = torch.zeros_like(q), torch.zeros_like(k)
    pa.pa_rope(a, b, q, k, pos, turns, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, want_q) and torch.equal(b, want_k)
    graph = torch.cuda.CUDAGraph()
    a.zero_(), b.zero_()
    with torch.cuda.graph(graph):
        pa.pa_rope(a, b, q, k, pos, turns)
    pos.add_(5)
    graph.replay()
    pa.pa_rope(want_q, want_k, q, k, pos, turns)
    torch.cuda.synchronize()
    assert torch.equal(a, want_q) and torch.equal(b, want_k)
