"""The rotary positions, the beam selection and the beams' reordering in 64 bits, plainly.

Written from the definitions in include/pa.h; shares nothing with the kernels or the binding."""
from fractions import Fraction
import math

import numpy as np


def frequencies(rotary, base=10000.0, scaling="none", factor=1.0, original_len=0, low=None, high=None):
    """(angle per position of every pair, attention factor)."""
    f = [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    m = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "ntk":
        wide = base * factor ** (rotary / (rotary - 2.0))
        f = [wide ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    elif scaling == "bands":
        low, high = low or 1.0, high or 4.0
        out = []
        for x in f:
            wave = 2 * math.pi / x
            if wave < original_len / high:
                out.append(x)
            elif wave > original_len / low:
                out.append(x / factor)
            else:
                r = (original_len / wave - low) / (high - low)
                out.append((1 - r) * x / factor + r * x)
        f = out
    elif scaling == "yarn":
        low, high = low or 1.0, high or 32.0

        def pair(turns):
            return rotary * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
        a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rotary - 1)
        out = []
        for i, x in enumerate(f):
            r = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            out.append(x / factor * r + x * (1 - r))
        f = out
        if factor > 1:
            m = 0.1 * math.log(factor) + 1
    return np.array(f), m


def rotate(x, positions, f, interleaved=False, m=1.0, inverse=False):
    """x [T, heads, hd] (float64), each pair turned by its angle; angles are reduced as exact
    integers times f in extended steps of 2^20 positions, so that far positions stay exact."""
    x = np.asarray(x, np.float64)
    n = len(f)
    pos = np.asarray(positions, np.int64)
    hi, lo = np.divmod(pos, 1 << 20)
    step = np.remainder(np.float64(1 << 20) * f, 2 * np.pi)
    a = hi[:, None].astype(np.float64) * step + lo[:, None].astype(np.float64) * f
    a = (-a if inverse else a)[:, None]
    y = x.copy()
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., i] = m * (x[..., i] * np.cos(a) - x[..., j] * np.sin(a))
    y[..., j] = m * (x[..., j] * np.cos(a) + x[..., i] * np.sin(a))
    return y


def rotation_slack(x, n, interleaved, m=1.0):
    """What fp32 may lose of each result: cos and sin are off by pi 2^-25 (the angle) and two units
    of 2^-24 each, the two products and the sum by 2^-24: under 2^-21 of |x1| + |x2| in all."""
    x = np.abs(np.asarray(x, np.float64))
    out = np.zeros_like(x)
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    out[..., i] = out[..., j] = (x[..., i] + x[..., j]) * abs(m) * 2.0 ** -21
    return out


def scores(logits, cum):
    """(cum + log_softmax of one beam in 64 bits, -inf where there is nothing; its largest logit; what
    x minus that has added to it)."""
    x = np.asarray(logits, np.float64)
    if cum == -np.inf or not (x > -np.inf).any():
        return np.full(x.shape, -np.inf), 0.0, 0.0
    top = x.max()
    with np.errstate(under="ignore"):
        offset = float(cum) - math.log(np.exp(x - top).sum())
    return (x - top) + offset, top, offset


def select(logits, cum, num_out, finished=None, end_token=0):
    """logits [R * B, V], cum [R, B] -> scores, beams, tokens [R, num_out], and the smallest
    difference of two unequal scores of different beams that decided an order.  The order is that of the
    exact sums: 64 bits drop an offset of 15 next to a logit of 1e29."""
    R, B = cum.shape
    V = logits.shape[1]
    sc = np.full((R, num_out), -np.inf)
    bm, tk = np.full((R, num_out), -1, np.int32), np.full((R, num_out), -1, np.int32)
    closest = np.inf
    for r in range(R):
        found = []
        for b in range(B):
            if finished is not None and finished[r, b]:
                if cum[r, b] > -np.inf:
                    found.append((-Fraction(float(cum[r, b])), b, end_token))
                continue
            x = logits[r * B + b]
            s, top, offset = scores(x, cum[r, b])
            with np.errstate(over="ignore"):
                s = np.where(s.astype(np.float32) > -np.inf, s, -np.inf)
            k = min(num_out + 1, V)
            floor = np.partition(s, V - k)[V - k]
            at = np.nonzero((s >= floor) & (s > -np.inf))[0]
            found += [(Fraction(float(top)) - Fraction(float(x[t])) - Fraction(offset), b, int(t)) for t in at]
        found.sort()
        for i in range(1, min(len(found), num_out + 1)):
            if found[i][1] != found[i - 1][1] and found[i][0] != found[i - 1][0]:
                closest = min(closest, float(found[i][0] - found[i - 1][0]))
        for i, (s, b, t) in enumerate(found[:num_out]):
            sc[r, i], bm[r, i], tk[r, i] = -float(s), b, t
    return sc, bm, tk, closest


def reorder(pools, tables, lens, parents, layout="HND"):
    """New (pools, tables) as copies; pools are arrays [blocks, ...], parents [R, B]."""
    old, new = [np.array(p) for p in pools], [np.array(p) for p in pools]
    R, B = parents.shape
    was, tables = np.array(tables), np.array(tables)
    for r in range(R):
        for j in range(B):
            p = parents[r, j]
            if p < 0 or p == j:
                continue
            a, c = r * B + p, r * B + j
            full, rest = divmod(int(lens[c]), 16)
            tables[c, :full] = was[a, :full]
            if rest:
                src, dst = was[a, full], was[c, full]
                for x, y in zip(old, new):
                    if layout == "HND":
                        y[dst, :, :rest] = x[src, :, :rest]
                    else:
                        y[dst, :rest] = x[src, :rest]
    return new, tables
