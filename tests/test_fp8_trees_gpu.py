"""Trees and wide page lists over 8-bit caches against bounds of the kernel's own precision.

With s the power of two that puts a row's largest |q s| in [128, 256), the pair of E4M3 values holds q s
exactly where |q s| >= 2^-2 (the first takes q's four leading bits, and what is left is at most eight
steps of the last of bf16's eight) and to half of E4M3's smallest step, 2^-10, elsewhere: |dq| <= 2^-17
max|q|.  So a score moves by at most e = scale 2^-17 max|q| sum_d |k_d|, a weight by a factor 1 +- e and
the normalisation by as much.  A weight is an f16 value (2^-11) in three E5M2 terms: nine bits, rounded
(2^-9, less than the 2^-8 that ref64's bound allows it), or half the smallest step, 2^-17, where the
row's largest is at least 2^7: over n keys of values like one another 2^-24 n of sum p |v|, taken
four times for values that are not alike."""
import math

import pytest
import torch

import paged_kv_gqa_15_gb300 as pa
from tests import ref64
from tests import test_pages_gpu as P
from tests import test_tree_gpu as T

DEV = "cuda"
gpu = pytest.mark.gpu


def extra(q, k, scale, kv_scale, n):
    """What the 8-bit path adds to ref64's relative room, from the inputs."""
    keys = k.view(torch.uint8).view(torch.float8_e4m3fn).float().nan_to_num(0.0).abs().sum(-1).max().item() * kv_scale
    return 2 * scale * 2.0 ** -17 * q.float().abs().max().item() * keys + 2.0 ** -11 + 2.0 ** -22 * n


def reference(c, window=0, q=None):
    rows = int(c["indptr"][-1])
    q = c["q"] if q is None else q
    return ref64.tree(q[:rows].cpu(), c["k"], c["v"], c["table"].cpu(), c["lens"].cpu(), c["indptr"].cpu(), c["mask"].cpu(),
                      c["scale"], c["layout"], window, c["kv_scale"], c["kv_scale"])


def room(c):
    return extra(c["q"], c["k"], c["scale"], c["kv_scale"], int(c["lens"].max()))


def first_code(q):
    """q without the second E4M3 value of the pair."""
    s = 2.0 ** (7 - torch.floor(torch.log2(q.float().abs().amax(-1, keepdim=True))))
    return ((q.float() * s).to(torch.float8_e4m3fn).float() / s).to(torch.bfloat16)


def slices(n, seed, hd=64, nodes=3, nq=3):
    """One long sequence.  Channel d of its values is 8 in the d-th stretch of keys and 0 elsewhere, so
    that an output channel is one stretch's share of the weights: whatever piece is lost, doubled or
    put elsewhere shows, and all terms have one sign (sum p |v| is the output itself)."""
    c = T.make([n], [nodes], nq, 1, hd, seed=seed, fp8=True)
    c["kv_scale"] = 1.0
    c["k"] = (c["k"].float() / 32).to(torch.float8_e4m3fn)
    v = torch.zeros(c["v"].shape)
    for t in range(n):
        v[c["table"][0, t // 16], :, t % 16, t * hd // n] = 8.0
    c["v"] = v.to(torch.float8_e4m3fn)
    return c


@gpu
@pytest.mark.parametrize("i", range(len(T.CASES)))
def test_trees_within_the_kernels_own_precision(i):
    lens, nodes, nq, nkv, hd = T.CASES[i]
    c = T.gpu(T.make(lens, nodes, nq, nkv, hd, seed=200 + i, fp8=True, layout="NHD" if i % 2 else "HND"))
    out, bound = reference(c)
    ref64.assert_attention(T.call(c), out, bound, room(c), str(T.CASES[i]))


@gpu
@pytest.mark.parametrize("hd,nq,nodes", [(64, 3, 3), (128, 8, 20), (256, 2, 5), (128, 4, 40)])
def test_every_piece_of_a_long_sequence_counts(hd, nq, nodes):
    c = T.gpu(slices(9000 + nodes, 90 + hd, hd, nodes, nq))
    out, bound = reference(c)
    ref64.assert_attention(T.call(c), out, bound, room(c))
    assert pa.device_status() == 0


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_what_the_bound_of_a_long_sequence_rejects(hd):
    """Zeros, a result without one of a hundred pieces, and weights of q's first code alone."""
    c = slices(9003, 90 + hd, hd)
    out, bound = reference(c)
    e = room(c)
    ref64.assert_attention(out.to(torch.bfloat16), out, bound, e)
    wrong = [torch.zeros_like(out)]
    for piece in (0, 37, 99):
        gone = out.clone()
        share = torch.zeros(hd)
        share[piece * hd // 100] = min(1.0, hd / 100)
        gone = gone * (1 - share)
        wrong.append(gone / (gone.sum(-1, keepdim=True) / 8))
    wrong.append(reference(c, q=first_code(c["q"]))[0])
    for x in wrong:
        with pytest.raises(AssertionError):
            ref64.assert_attention(x.to(torch.bfloat16), out, bound, e)


@pytest.mark.parametrize("i", [2, 3, 6])
def test_what_the_bound_of_the_trees_rejects(i):
    lens, nodes, nq, nkv, hd = T.CASES[i]
    c = T.make(lens, nodes, nq, nkv, hd, seed=200 + i, fp8=True, layout="NHD" if i % 2 else "HND")
    out, bound = reference(c)
    for x in (torch.zeros_like(out), reference(c, q=first_code(c["q"]))[0]):
        with pytest.raises(AssertionError):
            ref64.assert_attention(x.to(torch.bfloat16), out, bound, room(c))


@gpu
@pytest.mark.parametrize("far", [64.0, 1024.0, 8192.0])
def test_a_query_channel_far_above_the_others(far):
    """The keys are zero in that channel, so that the others decide; their error is that of the bound,
    2^-17 of the far one."""
    for hd in (64, 128, 256):
        c = T.make([300, 41], [9, 4], 8, 2, hd, seed=92, fp8=True)
        c["q"][..., 5] = far
        code = c["k"].view(torch.uint8)
        code[..., 5] = 0
        c = T.gpu(c)
        out, bound = reference(c)
        ref64.assert_attention(T.call(c), out, bound, room(c), f"{hd} {far}")


@gpu
@pytest.mark.parametrize("nq,nkv,hd", [(16, 1, 256), (10, 2, 256), (24, 2, 64), (17, 1, 64)])
@pytest.mark.parametrize("lens,most", [([1500, 40, 0, 977], 37), ([9000, 20, 0, 5007], 301)])
def test_wide_page_lists_within_the_kernels_own_precision(lens, most, nq, nkv, hd):
    c = P.make(lens, nq, nkv, hd, 93, True)
    P.fill_bounds(c)
    pages, kept = P.select(c, most, 1, 1)
    out, bound = ref64.decode_pages(c["q"], c["k"], c["v"], pages.cpu(), kept.cpu(), c["scale"], "HND", c["kv_scale"], c["kv_scale"])
    ref64.assert_attention(P.decode(c, pages, kept), out, bound,
                           extra(c["q"], c["k"], c["scale"], c["kv_scale"], most * 16))


@gpu
def test_weights_are_rounded_and_not_cut():
    """One key of weight 1 and 199 of e^-x = 1 - 2^-11, whose f16 value 128 (1 - 2^-11) has eleven ones: cut
    to nine bits it loses 0.1875 (2^-9.4 of its value), rounded it gains 0.0625.  All values are one
    number, 64 of them in a row over a step of bf16, so that the outputs' own rounding averages out
    to a 64th of a step: the mean of the outputs is off by at most half a step of nine bits just
    under 128, 2^-10, and that."""
    c = T.make([200], [1], 4, 1, 64, seed=94, fp8=True)
    c["q"] = torch.zeros_like(c["q"])
    c["q"][..., 0] = 1.0
    k = torch.zeros(c["k"].shape)
    k[c["table"][0, 3], :, 5, 0] = 1.0
    c["k"], c["v"] = k.to(torch.float8_e4m3fn), torch.ones(c["v"].shape).to(torch.float8_e4m3fn)
    c = T.gpu(c)
    scale = -math.log1p(-2.0 ** -11)
    off = []
    for i in range(64):
        value = 1.0 + (i + 0.5) / 64 * 2.0 ** -7
        out = torch.empty_like(c["q"])
        pa.pa_tree_decode(out, c["q"], c["k"], c["v"], c["table"], c["lens"], c["indptr"], c["mask"], scale, 1, T.space(c),
                          k_scale=1.0, v_scale=value)
        off.append(float(out.double().mean()) / value - 1.0)
    assert abs(sum(off) / 64) <= 2.0 ** -10 + 2.0 ** -7 / 64
