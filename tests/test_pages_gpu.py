"""Page bounds, page selection and the decode over selected pages against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa
from tests import ref64

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAGE = 16


def make(lens, nq, nkv, hd, seed, fp8=False, layout="HND", spread=1.0):
    rng = np.random.default_rng(seed)
    need = [(n + PAGE - 1) // PAGE for n in lens]
    nb = sum(need) + 3
    table = np.full((len(lens), max(max(need), 1)), np.iinfo(np.int32).max, np.int32)
    perm, at = rng.permutation(nb), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    gen = torch.Generator().manual_seed(seed)
    dims = (nb, nkv, PAGE, hd) if layout == "HND" else (nb, PAGE, nkv, hd)
    drift = torch.randn((nb, nkv, 1, hd) if layout == "HND" else (nb, 1, nkv, hd), generator=gen)
    scale = 1.0 / 32 if fp8 else 1.0
    k = torch.randn(dims, generator=gen) + spread * drift
    v = torch.randn(dims, generator=gen)
    for b, n in enumerate(lens):                       # rows past the sequence hold NaN
        for t in range(n, need[b] * PAGE):
            for x in (k, v):
                x[(table[b, t // PAGE], slice(None), t % PAGE) if layout == "HND" else
                  (table[b, t // PAGE], t % PAGE)] = math.nan
    k, v = ((x / scale).to(torch.float8_e4m3fn) if fp8 else x.to(torch.bfloat16) for x in (k, v))
    q = torch.randn(len(lens), nq, hd, generator=gen).to(torch.bfloat16)
    return dict(q=q.to(DEV), k=k.to(DEV), v=v.to(DEV), table=torch.from_numpy(table).to(DEV),
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), layout=layout, nkv=nkv, kv_scale=scale,
                bounds=torch.zeros((nb, nkv, 2, hd), dtype=k.dtype, device=DEV), scale=1.0 / math.sqrt(hd))


def fill_bounds(c, first=None, new=None):
    pa.pa_page_bounds(c["bounds"], c["k"], c["table"], c["lens"],
                      int(c["lens"].max()) if new is None else new, first_tokens=first, layout=c["layout"])


def select(c, most, sink=0, recent=1, ws=None, out=None):
    B = len(c["lens"])
    pages, lens = out or (torch.full((B, c["nkv"], most), -7, dtype=torch.int32, device=DEV),
                          torch.full((B,), -7, dtype=torch.int32, device=DEV))
    ws = pa.alloc_workspace(pa.select_pages_workspace_size(B, c["nkv"], c["table"].shape[1]), DEV) if ws is None else ws
    pa.pa_select_pages(pages, lens, c["q"], c["bounds"], c["table"], c["lens"], ws, sink_pages=sink, recent_pages=recent)
    return pages, lens


def check_select(c, most, sink=0, recent=1):
    pages, lens = select(c, most, sink, recent)
    want = ref64.select(c["q"], c["bounds"], c["table"].cpu(), c["lens"].cpu(), most, sink, recent)
    assert torch.equal(lens.cpu(), want[1])
    assert torch.equal(pages.cpu(), want[0])
    return pages, lens


def decode_space(c, most):
    return pa.alloc_workspace(pa.decode_split_workspace_size(*c["q"].shape, most * PAGE), DEV)


def decode(c, pages, lens, ws=None):
    out = torch.full_like(c["q"], math.nan)
    pa.pa_decode_pages(out, c["q"], c["k"], c["v"], pages, lens, c["scale"],
                       decode_space(c, pages.shape[2]) if ws is None else ws,
                       layout=c["layout"], k_scale=c["kv_scale"], v_scale=c["kv_scale"])
    return out


# the 8-bit tensor-core decode carries q to 2^-8 of its value and p to 2^-8: a score moves by at
# most 2^-8 sum |q k| scale (under 16 here), its weight by 0.065 and the sum by as much
FP8_EXTRA = 0.14


def same(a, b):
    a, b = (x.cpu().double() if x.dtype == torch.float64 else x.cpu().float().double() for x in (a, b))
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(0), b.nan_to_num(0))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_bounds_of_every_page(hd, layout, fp8):
    c = make([1, 16, 17, 0, 250, 31], 4, 2, hd, hd, fp8, layout)
    fill_bounds(c)
    zero = torch.zeros_like(c["bounds"])
    assert same(c["bounds"], ref64.bounds(zero, c["k"], c["table"].cpu(), c["lens"].cpu(), [0] * 6, layout))
    assert pa.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_bounds_of_new_tokens_only(fp8):
    c = make([33, 48, 70, 5, 100, 64], 3, 3, 128, 9, fp8)
    first = torch.tensor([32, 48, 30, 0, 99, 10], dtype=torch.int32, device=DEV)
    before = c["bounds"]
    want = ref64.bounds(before, c["k"], c["table"].cpu(), c["lens"].cpu(), first, "HND")
    fill_bounds(c, first, new=54)
    assert same(c["bounds"], want)
    assert pa.device_status() == 0


def test_bounds_of_as_many_new_tokens_as_there_may_be():
    c = make([33, 70], 3, 3, 128, 19)
    first = torch.tensor([16, 30], dtype=torch.int32, device=DEV)
    want = ref64.bounds(c["bounds"], c["k"], c["table"].cpu(), c["lens"].cpu(), first, "HND")
    fill_bounds(c, first, new=2 ** 31 - 1)
    assert same(c["bounds"], want)
    fill_bounds(c, new=2 ** 31 - 1)
    assert same(c["bounds"], ref64.bounds(want, c["k"], c["table"].cpu(), c["lens"].cpu(), [0, 0], "HND"))
    assert pa.device_status() == 0


def test_bounds_hand_nan_and_infinities_on():
    c = make([40], 2, 2, 64, 10)
    page = int(c["table"][0, 1])
    c["k"][page, 0, 3, 5], c["k"][page, 1, 7, 6], c["k"][page, 1, 0, 9] = math.nan, math.inf, -math.inf
    fill_bounds(c)
    assert same(c["bounds"], ref64.bounds(torch.zeros_like(c["bounds"]), c["k"], c["table"].cpu(), c["lens"].cpu(), [0], "HND"))


def test_bounds_flag_what_they_cannot_cover():
    c = make([100, 60], 2, 2, 64, 11)
    fill_bounds(c, new=50)                      # 100 tokens from the start
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
    c["table"][1, 2] = c["k"].shape[0]
    before = c["bounds"].clone()
    fill_bounds(c)
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
    c["table"][1, 2] = -1
    c["bounds"].copy_(before)
    fill_bounds(c)
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
    c["lens"][0] = 10 ** 6                       # more tokens than the table holds
    c["table"][1, 2] = 0
    fill_bounds(c, new=10 ** 6)
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS


SELECT = [
    # lens, nq, nkv, hd, most, sink, recent
    ([1, 15, 16, 17], 4, 2, 64, 1, 0, 1),
    ([500, 33, 0, 320], 8, 2, 128, 8, 1, 2),
    ([700, 701, 64], 7, 1, 128, 5, 2, 3),            # nothing left to choose
    ([2000, 999], 32, 2, 128, 33, 3, 5),
    ([1500], 3, 3, 256, 40, 0, 1),
    ([17000, 18000], 4, 1, 64, 300, 1, 1),           # more pages than a CTA has threads
    ([400], 40, 2, 64, 26, 1, 1),                    # one page fewer than there are
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("i", range(len(SELECT)))
def test_selection_is_exact(i, fp8):
    lens, nq, nkv, hd, most, sink, recent = SELECT[i]
    c = make(lens, nq, nkv, hd, 40 + i, fp8)
    fill_bounds(c)
    check_select(c, most, sink, recent)
    assert pa.device_status() == 0


def test_selection_in_a_table_wider_than_its_sequences():
    """Tables of 50000 entries, whose scores no longer fit shared memory."""
    c = make([3000, 700], 8, 2, 64, 47)
    fill_bounds(c)
    want = ref64.select(c["q"], c["bounds"], c["table"].cpu(), c["lens"].cpu(), 20, 1, 2)
    wide = torch.full((2, 50000), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
    wide[:, :c["table"].shape[1]] = c["table"]
    c["table"] = wide
    pages, lens = select(c, 20, 1, 2)
    assert torch.equal(pages.cpu(), want[0]) and torch.equal(lens.cpu(), want[1])
    assert pa.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_equal_scores_go_to_the_lower_page(fp8):
    c = make([1600, 800], 8, 2, 128, 50, fp8)
    fill_bounds(c)
    c["bounds"].copy_(c["bounds"][:1].expand_as(c["bounds"]).clone())       # every page alike
    check_select(c, 20, 1, 2)
    # two kinds of pages, the better ones fewer and more than are wanted
    for share in (3, 30):
        c["bounds"].copy_(c["bounds"][:1].expand_as(c["bounds"]).clone())
        c["bounds"][torch.arange(c["bounds"].shape[0], device=DEV) % share == 0] = \
            (c["bounds"][:1].float() + 0.5).to(c["bounds"].dtype)
        check_select(c, 20, 1, 2)


def test_pages_that_32_bits_cannot_tell_apart():
    """Scores of about 2^20 that differ by 2^-8: below half a step of fp32 at that size."""
    hd = 128
    c = make([1600], 1, 1, hd, 51)
    c["q"].zero_()
    c["q"][0, 0, :2] = torch.tensor([1024.0, 1.0])
    rng = np.random.default_rng(1)
    value = torch.zeros(c["bounds"].shape[0], dtype=torch.float32)
    value[c["table"][0, :100].long().cpu()] = torch.from_numpy(rng.permutation(100).astype(np.float32)) * 2.0 ** -8
    c["bounds"].zero_()
    c["bounds"][:, 0, :, 0] = 1024.0
    c["bounds"][:, 0, :, 1] = value.to(torch.bfloat16).to(DEV)[:, None]
    check_select(c, 30, 0, 1)


@pytest.mark.parametrize("most", [21, 25, 30])
def test_a_few_pages_at_the_border_that_32_bits_cannot_tell_apart(most):
    """20 pages above, 200 below, and 12 between whose scores differ below half a step of fp32."""
    c = make([233 * 16], 1, 1, 128, 55)
    c["q"].zero_()
    c["q"][0, 0, :2] = torch.tensor([1024.0, 1.0])
    rng = np.random.default_rng(3)
    kind = rng.permutation(232)
    first = np.where(kind < 20, 1200.0, np.where(kind < 32, 1024.0, 16.0 + 4 * (kind % 50)))
    second = np.where((kind >= 20) & (kind < 32), kind * 2.0 ** -8, 0.0)
    ids = c["table"][0, :232].long()
    c["bounds"].zero_()
    for d, x in ((0, first), (1, second)):
        c["bounds"][ids, 0, :, d] = torch.from_numpy(x).to(torch.bfloat16).to(DEV)[:, None]
    check_select(c, most, 0, 1)


def test_more_sequences_than_a_launch_scores():
    rng = np.random.default_rng(4)
    c = make([int(n) for n in rng.integers(0, 120, 1100)], 2, 1, 64, 56)
    fill_bounds(c)
    check_select(c, 3, 1, 1)
    assert pa.device_status() == 0


def test_products_below_the_normal_numbers():
    """Products of about 2^-142, of which fp32 keeps seven bits."""
    c = make([1600, 1440], 4, 2, 64, 54)
    c["q"] *= 2.0 ** -70
    c["k"] *= 2.0 ** -72
    fill_bounds(c)
    for most in (10, 30, 60):
        check_select(c, most, 0, 1)


def test_scores_that_are_not_finite():
    c = make([1600, 1600], 4, 2, 64, 52)
    fill_bounds(c)
    ids = c["table"][0].long()
    c["bounds"][ids[7], 0, 1, 3] = math.nan
    c["bounds"][ids[9], 1, 1, 4] = math.inf
    c["bounds"][ids[11], 1, 0, 4] = -math.inf
    c["q"][1, 0, 5] = 0.0
    check_select(c, 12, 1, 1)
    c["bounds"][c["table"][1].long(), 0, 1, 5] = math.inf        # no head of kv head 0 of ...
    c["q"][1, :2, 5] = 0.0                                        # ... sequence 1 weighs it
    check_select(c, 12, 1, 1)
    c["q"][0] = math.nan                                          # every page the largest
    check_select(c, 12, 0, 1)


def test_selection_flags_bad_pages_and_lengths():
    c = make([800, 800], 4, 2, 64, 53)
    fill_bounds(c)
    c["table"][0, 5], c["table"][1, 6] = -3, c["k"].shape[0]
    check_select(c, 12, 1, 1)
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
    c["lens"][1] = 10 ** 6
    select(c, 12)
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nq,nkv,hd", [(2, 2, 64), (8, 2, 64), (8, 2, 128), (7, 1, 128), (16, 1, 128),
                                       (24, 1, 128), (4, 4, 128), (6, 2, 256), (17, 1, 64)])
def test_decode_over_selected_pages(nq, nkv, hd, fp8):
    c = make([1500, 40, 0, 977], nq, nkv, hd, nq + hd, fp8, "NHD" if nq % 2 else "HND")
    fill_bounds(c)
    pages, lens = check_select(c, 37, 1, 2)
    got = decode(c, pages, lens)
    out, bound = ref64.decode_pages(c["q"], c["k"], c["v"], pages.cpu(), lens.cpu(), c["scale"], c["layout"],
                                    c["kv_scale"], c["kv_scale"])
    ref64.assert_attention(got, out, bound, FP8_EXTRA if fp8 else 0.0)
    assert bool((got[2] == 0).all())
    assert pa.device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nq,nkv,hd", [(8, 2, 256), (16, 1, 256), (10, 2, 256), (24, 2, 64), (17, 1, 64), (16, 2, 64)])
@pytest.mark.parametrize("lens,most", [([1500, 40, 0, 977], 37), ([9000, 20, 0, 5007], 301), ([7000], 400), ([33] * 3, 2)])
def test_decode_over_lists_of_wide_groups(lens, most, nq, nkv, hd, fp8):
    c = make(lens, nq, nkv, hd, nq + hd + most, fp8, "NHD" if nq % 4 else "HND")
    fill_bounds(c)
    pages, kept = select(c, most, 1, 1)
    got = decode(c, pages, kept)
    out, bound = ref64.decode_pages(c["q"], c["k"], c["v"], pages.cpu(), kept.cpu(), c["scale"], c["layout"],
                                    c["kv_scale"], c["kv_scale"])
    ref64.assert_attention(got, out, bound, FP8_EXTRA if fp8 else 0.0)
    assert bool((got[c["lens"] == 0] == 0).all())
    # no byte behind the workspace it asks for is written
    need = pa.decode_split_workspace_size(len(lens), nq, hd, most * PAGE)
    room = torch.full((need + 4096,), 171, dtype=torch.uint8, device=DEV)
    assert torch.equal(decode(c, pages, kept, room[:need]), got)
    assert bool((room[need:] == 171).all())
    assert pa.device_status() == 0


def test_decode_over_lists_of_more_sequences_than_a_launch():
    rng = np.random.default_rng(6)
    c = make([int(n) for n in rng.integers(0, 200, 1000)], 4, 1, 256, 62)
    fill_bounds(c)
    pages, kept = select(c, 9, 1, 1)
    out, bound = ref64.decode_pages(c["q"], c["k"], c["v"], pages.cpu(), kept.cpu(), c["scale"], c["layout"],
                                    c["kv_scale"], c["kv_scale"])
    ref64.assert_attention(decode(c, pages, kept), out, bound)
    assert pa.device_status() == 0


def test_wide_groups_flag_bad_page_lists():
    c = make([500, 300], 8, 2, 256, 63)
    fill_bounds(c)
    pages, lens = select(c, 16, 1, 1)
    pages[0, 1, 3], pages[1, 0, 2] = c["k"].shape[0], -5
    assert torch.isfinite(decode(c, pages, lens)).all()
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS
    pages, lens = select(c, 16, 1, 1)
    lens[1] = 10 ** 6
    decode(c, pages, lens)
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS


def test_all_pages_selected_is_the_split_decode():
    c = make([1500, 40, 977], 8, 2, 128, 60)
    fill_bounds(c)
    pages, lens = select(c, 94, 0, 1)
    ws = pa.alloc_workspace(pa.decode_split_workspace_size(3, 8, 128, 1500), DEV)
    want = torch.empty_like(c["q"])
    pa.pa_decode_split(want, c["q"], c["k"], c["v"], c["table"], c["lens"], c["scale"], 1500, ws)
    assert torch.equal(decode(c, pages, lens), want)


def test_decode_flags_bad_page_lists():
    c = make([500], 8, 2, 128, 61)
    fill_bounds(c)
    pages, lens = select(c, 16, 1, 1)
    pages[0, 1, 3] = c["k"].shape[0]
    assert torch.isfinite(decode(c, pages, lens)).all()
    assert pa.device_status() == 1 << pa.PA_ERR_DEVICE_BOUNDS


def test_steps_of_a_growing_sequence_captured_and_replayed():
    """Write, bounds of the new page, select, decode, as one captured step, over page borders."""
    c = make([400, 170], 8, 2, 128, 62)
    c["k"], c["v"] = c["k"].nan_to_num(0.0), c["v"].nan_to_num(0.0)
    spare = torch.cat([c["table"][:, :], torch.full((2, 3), 2 ** 31 - 1, dtype=torch.int32, device=DEV)], 1)
    spare[0, 25], spare[1, 11] = [int(i) for i in set(range(c["k"].shape[0])) - set(
        c["table"][0, :25].tolist() + c["table"][1, :11].tolist())][:2]
    c["table"] = spare.contiguous()
    fill_bounds(c)
    gen = torch.Generator().manual_seed(3)
    kn, vn = (torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots, first = torch.zeros(2, dtype=torch.int64, device=DEV), c["lens"].clone()
    most = 9
    out = (torch.empty((2, 2, most), dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV))
    ws = pa.alloc_workspace(pa.select_pages_workspace_size(2, 2, c["table"].shape[1]), DEV)
    ws2 = decode_space(c, most)
    o = torch.empty_like(c["q"])

    def step():
        pa.pa_write_cache(kn, vn, c["k"], c["v"], slots)
        pa.pa_page_bounds(c["bounds"], c["k"], c["table"], c["lens"], 1, first_tokens=first)
        select(c, most, 1, 1, ws, out)
        pa.pa_decode_pages(o, c["q"], c["k"], c["v"], out[0], out[1], c["scale"], ws2)

    def advance():
        first.copy_(c["lens"])
        for b in range(2):
            n = int(c["lens"][b])
            slots[b] = int(c["table"][b, n // PAGE]) * PAGE + n % PAGE
        c["lens"] += 1
        kn.copy_(torch.randn(2, 2, 128, generator=gen)), vn.copy_(torch.randn(2, 2, 128, generator=gen))
        c["q"].copy_(torch.randn(2, 8, 128, generator=gen))

    advance()
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(9):
        advance()
        graph.replay()
        torch.cuda.synchronize()
        want = ref64.select(c["q"], c["bounds"], c["table"].cpu(), c["lens"].cpu(), most, 1, 1)
        assert torch.equal(out[0].cpu(), want[0]) and torch.equal(out[1].cpu(), want[1])
        ref, bound = ref64.decode_pages(c["q"], c["k"], c["v"], out[0].cpu(), out[1].cpu(), c["scale"])
        ref64.assert_attention(o, ref, bound)
    fresh = torch.zeros_like(c["bounds"])
    kept, c["bounds"] = c["bounds"], fresh
    fill_bounds(c)
    used = torch.cat([c["table"][0, :26], c["table"][1, :12]]).long()
    assert same(kept[used], fresh[used])
    assert pa.device_status() == 0
