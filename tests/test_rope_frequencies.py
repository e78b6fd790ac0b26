"""The frequency tables against their definitions in 60 digits: every entry is the nearest multiple of 2^-64
of a turn, and the angle that the kernels take from it is held to 2^-24 of a half turn at positions up to 2^31."""
from decimal import Decimal, getcontext, localcontext
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")
UNIT = Decimal(2) ** 64
# entries come from arithmetic of twice 53 bits: under 2^-40 of a unit beside the half that rounding costs
ROOM = Decimal(1) / 2 + Decimal(2) ** -30
CASES = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="linear", factor=1 / 3), dict(scaling="ntk", factor=8.0),
         dict(scaling="ntk", factor=0.7), dict(scaling="bands", factor=8.0, original_len=8192),
         dict(scaling="bands", factor=2.5, original_len=100, low=0.5, high=7.0),
         dict(scaling="yarn", factor=32.0, original_len=4096), dict(scaling="yarn", factor=0.5, original_len=64, low=2.0, high=9.0),
         dict(scaling="yarn", factor=4.0, original_len=4, low=2.0, high=9.0)]      # a ramp of no width


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return pa.load()


def frequencies(rotary, base, scaling="none", factor=1.0, original_len=0, low=None, high=None):
    """Radians per position of every pair."""
    base, s, pairs = Decimal(base), Decimal(factor), rotary // 2
    if scaling == "ntk":
        base *= (s.ln() * rotary / (rotary - 2)).exp()
    f = [(base.ln() * -2 * i / rotary).exp() for i in range(pairs)]
    if scaling == "linear":
        f = [x / s for x in f]
    if scaling == "bands":
        low, high = Decimal(low or 1.0), Decimal(high or 4.0)
        part = [min(max((original_len * x / (2 * PI) - low) / (high - low), Decimal(0)), Decimal(1)) for x in f]
        f = [x * ((1 - r) / s + r) for x, r in zip(f, part)]
    if scaling == "yarn":
        def pair(turns):
            return rotary * (original_len / (Decimal(turns) * 2 * PI)).ln() / (2 * base.ln())
        a = max(math.floor(pair(high or 32.0)), 0)
        b = min(math.ceil(pair(low or 1.0)), rotary - 1)
        part = [min(max((i - a) / max(Decimal(b - a), Decimal(0.001)), Decimal(0)), Decimal(1)) for i in range(pairs)]
        f = [x * (r / s + 1 - r) for x, r in zip(f, part)]
    return f


def off(entry, f):
    """How far an entry is from f radians per position, in units."""
    d = (Decimal(int(entry) % (1 << 64)) - f / (2 * PI) * UNIT) % UNIT
    return min(abs(d), abs(UNIT - abs(d)))


def entries(turns):
    return [int(t) % (1 << 64) for t in turns]


@pytest.mark.parametrize("rotary", [2, 6, 100, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5, 1e300])
@pytest.mark.parametrize("scaling", CASES)
def test_entries_are_the_nearest(rotary, base, scaling):
    if rotary == 2 and scaling.get("scaling") == "ntk":
        return                                           # refused
    turns, _ = pa.rope_table(rotary, base, device="cpu", **scaling)
    # of bases beyond 2^900 a frequency has 53 bits, a few of them lost to its power
    rest = UNIT * Decimal(2) ** -48 if base > 2.0 ** 900 else 0
    for got, f in zip(entries(turns), frequencies(rotary, base, **scaling)):
        assert off(got, f) <= ROOM + rest * f


def test_entries_of_any_frequencies():
    rng = np.random.default_rng(3)
    f = [1.0, -1.0, 0.0, math.pi, 2 * math.pi, math.pi / 2, -7.25, 1e-30, 1e9, -3.7e15, 1.2e19, 2.0 ** 53 + 2, 5e-324]
    f += list(rng.standard_normal(60) * np.exp(rng.uniform(-30, 30, 60)))
    with localcontext() as more:
        more.prec = 90
        for got, x in zip(entries(pa.rope_table_of(f, device="cpu")), f):
            assert off(got, Decimal(float(x))) <= ROOM + abs(Decimal(float(x))) * UNIT * Decimal(10) ** -58, x


@pytest.mark.parametrize("base,scaling", [(10000.0, {}), (500000.0, {}), (1e6, dict(scaling="ntk", factor=8.0)),
                                          (10000.0, dict(scaling="linear", factor=0.3))])
def test_angles_of_far_positions(base, scaling):
    """The kernels' way from an entry to half turns (an integer product, its top 32 bits as fp32)."""
    rng = np.random.default_rng(4)
    turns, _ = pa.rope_table(128, base, device="cpu", **scaling)
    f = frequencies(128, base, **scaling)
    for p in [1 << 31, -(1 << 31), (1 << 31) - 1, 1, 0, 12345] + [int(x) for x in rng.integers(1 << 30, 1 << 31, 30)]:
        for got, x in list(zip(entries(turns), f))[::7] + [(entries(turns)[0], f[0])]:
            top = (got * p % (1 << 64)) >> 32
            half_turns = np.float32(top - (1 << 32) if top >> 31 else top) * np.float32(2.0 ** -31)
            d = (Decimal(float(half_turns)) - p * x / PI) % 2
            assert min(d, 2 - d) <= Decimal(2) ** -24, (p, x)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved,rotary", [(False, 128), (True, 128), (False, 100), (True, 38)])
def test_positions_next_to_whole_turns(interleaved, rotary):
    """Positions that are nearly whole turns of the first pair: its sine is the angle itself, which fp32 half
    turns hold to their last bits, so that an entry's own error shows."""
    pos = [103993, 312689, 4272943, 80143857, 411557987, 2 * 1068966896, 710]
    pos = pos + [-p for p in pos] + [44, 0]
    hd = 128
    x = torch.zeros((len(pos), 2, hd), dtype=torch.bfloat16, device="cuda")
    x[:, :, 0] = 1.0                                     # pair 0 is (1, 0), in either layout
    turns, _ = pa.rope_table(rotary)
    y = torch.empty_like(x)
    pa.pa_rope(y, None, x, None, torch.tensor(pos, device="cuda"), turns, interleaved=interleaved)
    got = y[:, 1, 1 if interleaved else rotary // 2].double().cpu().tolist()
    for p, s in zip(pos, got):
        a = Decimal(p) % (2 * PI)
        a = float(a - 2 * PI if a > PI else a + 2 * PI if a < -PI else a)
        # the top 32 bits of the turn are cut off, the entry is off by half a unit a position; then a few roundings
        # of 2^-24 and half a step of bf16
        room = math.pi * (2.0 ** -31 + abs(p) * 2.0 ** -64) + abs(math.sin(a)) * 2.0 ** -21
        assert abs(s - math.sin(a)) <= room + (abs(math.sin(a)) + room) * torch.finfo(torch.bfloat16).eps / 2, p
