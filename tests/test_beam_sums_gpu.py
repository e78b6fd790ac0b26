"""The log-sum-exp of pa_beam_select on rows made to gather its errors: mass at one distance below the top,
rows that rise from end to end (every group of chunks has a new maximum, in rows that one warp reads alone), stairs.

A row's cum is chosen so that its best score is next to 0, where fp32 shows the sum's own error.  The bound is the
documented 2^-17."""
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOUND = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()
    yield
    assert pa.device_status() == 0


class Search:
    """Rows out of the search but for one; R * B of them decide how many warps share a row."""

    def __init__(self, R, B, vocab, dtype):
        self.R, self.B = R, B
        self.logits = torch.zeros((R * B, vocab), dtype=dtype, device=DEV)
        self.cum = torch.full((R, B), -math.inf, device=DEV)
        self.space = pa.alloc_workspace(pa.beam_select_workspace_size(R, B, vocab), DEV)
        self.out = (torch.empty((R, 1), device=DEV), *(torch.empty((R, 1), dtype=torch.int32, device=DEV) for _ in range(2)))

    def error(self, x, captured=False):
        """x one row; how far cum + top - logsumexp is from that in 64 bits."""
        row = self.R * self.B // 2
        self.logits[row] = x
        y = self.logits[row].double()
        top = float(y.max())
        want = float(torch.log(torch.exp(y - top).sum()))
        cum = np.float32(want)
        self.cum.view(-1)[row] = float(cum)

        def call():
            pa.pa_beam_select(*self.out, self.logits, self.cum, self.space)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            graph.replay()
        else:
            call()
        token = int(self.out[2][row // self.B, 0])
        assert int(self.out[1][row // self.B, 0]) == row % self.B and float(y[token]) == top
        score = float(self.out[0][row // self.B, 0])
        return abs(score - (float(cum) - want)) - abs(score) * 2.0 ** -24


@pytest.mark.parametrize("R,B,V", [(1, 1, 260000), (1, 1, 1 << 24), (152, 32, 5000), (40, 8, 50257)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_peak_over_a_flat_row(R, B, V, dtype):
    s = Search(R, B, V, dtype)
    for low, d in [(5.4857059, 11.1170971), (6.614572, 11.973198), (-3.3, 8.0)] + \
            [(0.7, float(d)) for d in np.arange(8, 20, 0.37)] + [(-7.1, float(d)) for d in np.arange(20, 34, 2.1)]:
        for at in (7, V - 1, V // 2):
            x = torch.full((V,), low, device=DEV)
            x[at] = low + d
            assert s.error(x) <= BOUND, (low, d, at)


@pytest.mark.parametrize("R,B,V", [(152, 32, 131072), (77, 32, 1 << 20), (152, 32, 30001), (8, 8, 131072), (1, 1, 1 << 22)])
def test_rows_that_rise_from_end_to_end(R, B, V):
    s = Search(R, B, V, torch.float32)
    t = torch.arange(V, device=DEV, dtype=torch.float64)
    for span in (0.01, 0.02, 0.1, 0.3, 1.0, 3.0, 7.9, 8.1, 10.0, 16.5, 30.0, 100.0, 1000.0):
        x = (t * (span / V) - 3).float()
        assert s.error(x) <= BOUND, span
        assert s.error(x.flip(0)) <= BOUND, -span


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_stairs(dtype):
    """Steps of any height, each with mass enough to count beside the next ones."""
    for R, B, V in ((152, 32, 131072), (3, 4, 128001)):
        s = Search(R, B, V, dtype)
        rng = np.random.default_rng(5)
        for step in (0.25, 1.0, 4.0, 7.75, 8.0, 8.25, 9.0, 12.0, 20.0):
            for _ in range(3):
                # the last steps hold e^step times fewer logits each
                ends, left = [], V
                while left > 0:
                    ends.append(left)
                    left = int(left * (1 - 1 / (1.5 + rng.random() * math.exp(min(step, 9.0)))))
                    if len(ends) > 400:
                        break
                x = torch.zeros(V, device=DEV)
                for i, e in enumerate(reversed(ends)):
                    x[:e] -= step if i < len(ends) - 1 else 0
                assert s.error(x) <= BOUND, step
                x += 100 * float(rng.standard_normal())
                assert s.error(x, captured=True) <= BOUND, step


def test_large_logits_that_rise():
    s = Search(152, 32, 70000, torch.float32)
    t = torch.arange(70000, device=DEV, dtype=torch.float64)
    for slope, start in ((1.0, 2.0 ** 23), (1.0, -(2.0 ** 23) - 35000), (0.01, 2.0 ** 23 - 350), (3.0, 2.0 ** 24), (1e30, 0.0),
                         (16.0, 2.0 ** 27), (7e33, -2.4e38)):
        assert s.error((t * slope + start).float()) <= BOUND, (slope, start)


@pytest.mark.parametrize("R,B,V", [(1, 1, 1), (2, 3, 5000), (152, 32, 2000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_token_alone_keeps_its_beams_score(R, B, V, dtype):
    """log 1 is 0 without an error, whatever the logit."""
    s = Search(R, B, V, dtype)
    row = R * B // 2
    s.cum.view(-1)[row] = -13.7
    for value in (3.3, -50.1, 1e30, 0.0, float(torch.finfo(dtype).min)):
        s.logits[row] = -math.inf
        s.logits[row, V // 3] = value
        pa.pa_beam_select(*s.out, s.logits, s.cum, s.space)
        assert float(s.out[0][row // B, 0]) == float(np.float32(-13.7)) and int(s.out[2][row // B, 0]) == V // 3
