"""The E4M3 codes of turned keys where the two products that enclose a quotient have different codes, so that
pa_rope_append divides: those of pa_write_cache on the turned keys, bit for bit.

Angles are whole quarters of a turn, whose cosines and sines are 0 and 1, so that a turned key is a bf16 value: its
partner or itself, with either sign.  Each pair has quarters of its own, so that another pair's angle, another
partner or another sign is another code.  Scales are such that many keys lie next to a border between two codes."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build_library()
    yield
    assert pa.device_status() == 0


def scale_at(value, border):
    """An fp32 scale that is no power of two and takes `value` next to the border between two codes."""
    return float(np.float32(np.float64(value) / border))


def codes(x, factor):
    """Codes of fp32 products with an fp32 factor, by torch's conversion on the CPU."""
    y = x.float() * torch.tensor(factor, dtype=torch.float32)
    return y.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)


def divided(x, scale):
    """Whether products by factors 2^-21 under and over 1 / scale have different codes."""
    return codes(x, np.float32(1 / np.float64(scale) * (1 - 2.0 ** -21))) != codes(x, np.float32(1 / np.float64(scale) * (1 + 2.0 ** -21)))


def keys(tokens, heads, hd, scale, values, seed):
    """Half of the keys are `values` times powers of two, the rest any magnitude that has codes."""
    rng = np.random.default_rng(seed)
    shape = (tokens, heads, hd)
    x = rng.choice(values, shape) * 2.0 ** rng.integers(-10, 2, shape)
    x = np.where(rng.random(shape) < 0.5, x, rng.standard_normal(shape) * 2.0 ** rng.integers(-8, 10, shape) * scale)
    x = torch.from_numpy(x * rng.choice([-1.0, 1.0], shape)).to(torch.bfloat16)
    assert (x != 0).all()
    return x


def turned(x, quarters, interleaved):
    """x [T, heads, hd] with pair i turned by quarters [T, pairs] quarter turns."""
    n = quarters.shape[1]
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b, q, y = x[..., i], x[..., j], quarters[:, None, :], x.clone()
    for k, (c, d) in enumerate(((a, b), (-b, a), (-a, -b), (b, -a))):
        y[..., i] = torch.where(q == k, c, y[..., i])
        y[..., j] = torch.where(q == k, d, y[..., j])
    return y


# border: a half way between two codes; value: a bf16 number
SCALES = [(1.5, 17 / 16), (1.3046875, 19 / 16), (1.0078125, 29 / 16), (1.9921875, 25 / 16)]


def case(tokens, heads, hd, rotary, which):
    value, border = SCALES[which]
    ks = scale_at(value, border) / 64
    vs = scale_at(SCALES[which - 1][0], SCALES[which - 1][1]) / 32
    x = keys(tokens, heads, hd, ks, [value], 91 + which)
    v = keys(tokens, heads, hd, vs, [SCALES[which - 1][0]], 95 + which)
    rng = np.random.default_rng(99)
    per_position = torch.from_numpy(rng.integers(0, 4, rotary // 2))
    positions = torch.from_numpy(rng.integers(-(1 << 40), 1 << 40, tokens))
    return ks, vs, x, v, per_position, positions


LAYOUTS = [(64, 64, False), (128, 128, False), (128, 32, False), (256, 256, False), (256, 64, True), (128, 128, True),
           (64, 64, True), (128, 38, True), (64, 2, True), (64, 6, False), (128, 100, False), (256, 250, False)]


@pytest.mark.parametrize("which", range(len(SCALES)))
@pytest.mark.parametrize("hd,rotary,interleaved", LAYOUTS)
def test_the_keys_are_divided(hd, rotary, interleaved, which):
    """What the comparison below rests on, on the CPU: every second key's codes differ, in all channels."""
    ks, vs, x, v, per_position, positions = case(40, 2, hd, rotary, which)
    y = turned(x, (per_position * positions[:, None]) % 4, interleaved)
    often = divided(y, ks)
    assert 0.4 < often.float().mean() < 0.6 and 0.4 < divided(v, vs).float().mean() < 0.6
    assert (often.float().mean((0, 1)) > 0.2).all()
    # next to a border the quotient's code is the even one: the lower product's for some scales, else the upper's
    low = codes(y, np.float32(1 / np.float64(ks) * (1 - 2.0 ** -21)))
    q = (y.float() / torch.tensor(ks, dtype=torch.float32)).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
    assert ((q[often] == low[often]).float().mean() > 0.5) == (which in (0, 2, 3))


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(len(SCALES)))
@pytest.mark.parametrize("tokens,layout", [(40, "HND"), (3001, "NHD")])
@pytest.mark.parametrize("hd,rotary,interleaved", LAYOUTS)
def test_codes_of_divided_keys(built, tokens, layout, hd, rotary, interleaved, which):
    heads = 2
    ks, vs, x, v, per_position, positions = case(tokens, heads, hd, rotary, which)
    y = turned(x, (per_position * positions[:, None]) % 4, interleaved)
    assert divided(y, ks).sum() > tokens * hd // 2
    turns = torch.where(per_position < 2, per_position << 62, (per_position - 4) << 62)      # of 2^64 a turn
    blocks = tokens // 16 + 2
    shape = (blocks, heads, 16, hd) if layout == "HND" else (blocks, 16, heads, hd)
    got, want = [[torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2)] for _ in range(2)]
    slots = torch.from_numpy(np.random.default_rng(98).permutation(blocks * 16)[:tokens]).to(DEV)
    q = x.to(DEV)
    q_out = torch.empty_like(q)
    pa.pa_rope_append(q_out, q, q, v.to(DEV), *got, slots, positions.to(DEV), turns.to(DEV), layout=layout,
                      interleaved=interleaved, k_scale=ks, v_scale=vs)
    pa.pa_write_cache(y.to(DEV), v.to(DEV), *want, slots, layout=layout, k_scale=ks, v_scale=vs)
    assert torch.equal(q_out.cpu(), y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
