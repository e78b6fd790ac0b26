"""pa_beam_select against the selection in 64 bits (tests/rope_beam_ref.py).

Beams and tokens are equal, scores off by the 2^-20 that a row's log-sum-exp may be off and a
rounding to fp32.  Inputs have no two beams' candidates closer than that where their order counts
(looked at before the comparison), but for those that are equal by construction."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa
from tests import rope_beam_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NEAR = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()
    yield
    assert pa.device_status() == 0


def call(logits, cum, num_out, finished=None, end_token=0, space=None, out=None, stream=None):
    R, B = cum.shape
    if out is None:
        out = (torch.full((R, num_out), 7.0, device=DEV),
               *(torch.full((R, num_out), -7, dtype=torch.int32, device=DEV) for _ in range(2)))
    if space is None:
        space = pa.alloc_workspace(pa.beam_select_workspace_size(R, B, logits.shape[1]), DEV)
        space.fill_(0xA5)              # nothing in it has to be initialised
    pa.pa_beam_select(*out, logits, cum, space, finished=finished, end_token=end_token, stream=stream)
    return out


def check(logits, cum, num_out, finished=None, end_token=0, ties=False):
    """logits a CPU tensor; compares the call on its values."""
    x = logits.to(DEV) if logits.device.type == "cpu" else logits
    c = torch.from_numpy(np.asarray(cum, np.float32)).to(DEV)
    f = None if finished is None else torch.from_numpy(finished.astype(np.uint8)).to(DEV)
    got = call(x, c, num_out, f, end_token)
    sc, bm, tk, closest = ref.select(x.float().cpu().double().numpy(), np.asarray(cum, np.float32).astype(np.float64),
                                     num_out, finished, end_token)
    assert ties or closest > 2 * NEAR, "the inputs' order is not clear"
    assert np.array_equal(got[1].cpu().numpy(), bm)
    assert np.array_equal(got[2].cpu().numpy(), tk)
    s, none = got[0].cpu().double().numpy(), np.isinf(sc)
    assert np.array_equal(np.isinf(s), none) and (s[none] == -np.inf).all()
    assert (np.abs(s[~none] - sc[~none]) <= NEAR + np.abs(sc[~none]) * 2.0 ** -24).all()
    return got


def normal(rows, vocab, seed, dtype, scale=3.0):
    x = np.random.default_rng(seed).standard_normal((rows, vocab)) * scale
    return torch.from_numpy(x).to(dtype)


def spread_cum(R, B, seed):
    return -np.random.default_rng(seed).random((R, B)) * 4 - 10


DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,B,V,K", [
    (1, 1, 1, 1), (1, 1, 1, 3), (1, 4, 3, 8), (2, 2, 255, 4), (3, 1, 256, 1), (2, 3, 257, 6), (1, 32, 1000, 64),
    (5, 4, 8191, 8), (2, 5, 50001, 10), (3, 8, 32000, 16), (1, 2, 70000, 33), (2, 16, 4099, 32), (40, 4, 2048, 5),
    (1, 1, 262145, 64), (2, 7, 129, 17),
])
def test_plain(R, B, V, K, dtype):
    check(normal(R * B, V, R + B + V, dtype), spread_cum(R, B, V + K), K)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,stride", [(0, 1024), (1, 1024), (3, 1001), (8, 1008), (16, 1003)])
def test_rows_of_any_alignment(dtype, offset, stride):
    """Rows inside a wider buffer whose other values would win if they were read."""
    R, B, V = 3, 2, 997
    x = normal(R * B, V, 5, dtype)
    buffer = torch.full((offset + R * B * stride + 64,), 1e4, dtype=dtype, device=DEV)
    view = buffer[offset:].as_strided((R * B, V), (stride, 1))
    view.copy_(x)
    check(view, spread_cum(R, B, 6), 7)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [600, 20000])
def test_equal_rows_and_equal_logits(dtype, V):
    """Equal scores go to the lower beam, then to the lower token, however the rows are aligned."""
    R, B = 2, 4
    one = normal(1, V, 9, dtype)
    one[0, [5, 300, 511, V - 1]] = 9.5                    # the same largest logit four times
    x = one.expand(R * B, V).contiguous()
    check(x, np.full((R, B), -3.25), 14, ties=True)
    check(torch.zeros((R * B, V), dtype=dtype), np.full((R, B), -1.0), 64, ties=True)
    wide = torch.full((R * B, V + 1), 50.0, dtype=dtype, device=DEV)     # rows start at any element
    wide[:, :V] = x.to(DEV)
    check(wide[:, :V], np.full((R, B), -3.25), 14, ties=True)


def test_more_equal_chunks_than_are_ranked():
    for B, V, K in ((4, 300000, 16), (1, 1 << 20, 3), (32, 20000, 64)):
        check(torch.full((B, V), -2.5, dtype=torch.bfloat16), np.full((1, B), -1.0), K, ties=True)
        x = torch.full((B, V), -2.5, dtype=torch.float32)
        x[:, V // 2:] = -2.25                          # the better half: still too many
        check(x, np.full((1, B), -1.0), K, ties=True)


def test_first_step_finished_and_dead_beams():
    R, B, V, K = 4, 4, 3001, 8
    x = normal(R * B, V, 13, torch.float32)
    cum = spread_cum(R, B, 14)
    cum[0, 1:], cum[2, :] = -np.inf, -np.inf
    finished = np.zeros((R, B), bool)
    finished[1, [0, 3]] = finished[3, :] = finished[0, 2] = finished[2, 1] = True
    cum[1, 0], cum[1, 3] = -1.0, -17.0                    # ends first, and among the others or not at all
    poisoned = x.clone()                                  # rows that are not read
    for r in range(R):
        for b in range(B):
            if finished[r, b] or cum[r, b] == -np.inf:
                poisoned[r * B + b] = float("nan")
    got = check(x, cum, K, finished, 2)
    again = call(poisoned.to(DEV), torch.from_numpy(cum.astype(np.float32)).to(DEV), K,
                 torch.from_numpy(finished).to(DEV), 2)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    assert (got[1][2] == -1).all() and got[2][1, 0] == 2 and got[1][1, 0] == 0
    assert (got[2][3, :4] == 2).all() and (got[1][3, 4:] == -1).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_masks(dtype):
    """Rows with few tokens allowed, one or none; the type's lowest value in place of -inf."""
    R, B, V, K = 3, 3, 9000, 12
    x = normal(R * B, V, 21, dtype)
    rng = np.random.default_rng(22)
    low = torch.finfo(dtype).min
    for row in range(R * B):
        allowed = torch.from_numpy(rng.choice(V, [V, 40, 5, 1, 0, 3, 30, 2, 7][row], replace=False))
        keep = x[row, allowed].clone()
        x[row] = low if row in (6, 7) else -np.inf
        x[row, allowed] = keep
    check(x, spread_cum(R, B, 23), K)
    # a row of lowest values alone: every token is as good as another
    x[3:6] = low
    check(x, spread_cum(R, B, 24), K)
    x[:] = -np.inf
    got = check(x, spread_cum(R, B, 25), K)
    assert (got[1] == -1).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_offsets_and_magnitudes(dtype):
    """Logits shifted by a large number, widely spread ones, and accumulated scores of a long search."""
    x = normal(8, 5000, 31, torch.float32)
    for scale, shift, base in ((1.0, 3000.0, -10.0), (200.0, 0.0, -2.0), (1e30, 0.0, -2.0), (1.0, 0.0, -9000.0),
                               (1e-6, 0.0, -1.0)):
        y = (x * scale + shift).to(dtype)
        check(y, spread_cum(2, 4, 32) + base, 9, ties=scale != 200.0)


def test_candidates_that_few_threads_hold():
    """Chunks and elements laid out so that the best all lie with a few groups of threads, more than
    are ranked by counting: they are taken one by one."""
    rng = np.random.default_rng(41)
    B, V = 4, 1024 * 256                              # 1024 chunks a beam, one a thread
    x = rng.standard_normal((B, V)).astype(np.float32)
    x = x.reshape(B, 1024, 256)
    group = np.arange(1024) // 32
    x[:, group < 16] += 200 - 5 * group[group < 16][None, :, None].astype(np.float32)
    check(torch.from_numpy(x.reshape(B, V)), np.full((1, B), -2.0) - np.arange(B) * 0.01, 16)
    # the 16 chosen chunks: those at 0, 1 of every four full of high values, falling from group to
    # group of the threads that look at them, the others with one high value each
    x = np.full((1, 64, 256), -5.0, np.float32) + rng.random((1, 64, 256)).astype(np.float32)
    for s in range(16):
        chunk = 3 * s + 1
        x[0, chunk, 0] = 20.0 - s * 0.25
        if s % 4 < 2:
            e = np.arange(256)
            x[0, chunk] = 4 - 0.1 * ((s % 4) * 8 + e // 32) + 0.01 * rng.random(256)
            x[0, chunk, 0] = 20.0 - s * 0.25
    check(torch.from_numpy(x.reshape(1, -1)), np.zeros((1, 1)), 16)
    x[0, 1::3] += 30                                  # and with chunks that hold the maximum everywhere
    x[0, 1] = 60.0
    check(torch.from_numpy(x.reshape(1, -1)), np.zeros((1, 1)), 64)


def test_bad_rows_are_flagged():
    R, B, V = 3, 2, 700
    for bad, where in ((np.nan, 0), (np.inf, 0), (np.nan, 699), (np.inf, 350)):
        x = normal(R * B, V, 51, torch.float32)
        cum = spread_cum(R, B, 52)
        x[2, where] = bad
        got = call(x.to(DEV), torch.from_numpy(cum.astype(np.float32)).to(DEV), 4)
        assert pa.device_status() == 1 << pa.PA_ERR_INVALID
        out = cum.copy()
        out[1, 0] = -np.inf                           # the beam offers nothing
        x[2] = 0.0
        want = check(x, out, 4)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    for bad in (np.nan, np.inf):
        x = normal(R * B, V, 53, torch.float32)
        cum = spread_cum(R, B, 54)
        cum[0, 1] = bad
        got = call(x.to(DEV), torch.from_numpy(cum.astype(np.float32)).to(DEV), 4)
        assert pa.device_status() == 1 << pa.PA_ERR_INVALID
        cum[0, 1] = -np.inf
        for a, b in zip(got, check(x, cum, 4)):
            assert torch.equal(a, b)


def test_one_workspace_in_two_replayed_graphs_and_a_side_stream():
    R, B, V, K = 2, 4, 12345, 8
    a, b = normal(R * B, V, 61, torch.bfloat16).to(DEV), normal(R * B, V, 62, torch.float32).to(DEV)
    cum = torch.from_numpy(spread_cum(R, B, 63).astype(np.float32)).to(DEV)
    space = pa.alloc_workspace(pa.beam_select_workspace_size(R, B, V), DEV)
    want = [call(x, cum, K) for x in (a, b)]
    outs = [tuple(torch.zeros_like(t) for t in want[0]) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, x, out in zip(graphs, (a, b), outs):
        with torch.cuda.graph(g):
            call(x, cum, K, space=space, out=out)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(out, w))
    new = normal(R * B, V, 64, torch.bfloat16).to(DEV)
    want = call(new, cum, K)
    a.copy_(new)
    graphs[0].replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(b, cum, K, stream=side, space=space, out=tuple(torch.zeros_like(t) for t in outs[1]))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(outs[0], want))
    assert all(torch.equal(x, y) for x, y in zip(other, outs[1]))


def test_calls_on_two_streams_at_once():
    """Each with a workspace of its own; logits made and results taken by the kernels around the calls."""
    shapes = [(3, 4, 20011, torch.bfloat16), (40, 4, 20000, torch.float32)]
    sides, jobs = [torch.cuda.Stream() for _ in shapes], []
    for R, B, V, dtype in shapes:
        x = normal(R * B, V, R, dtype).to(DEV)
        cum = torch.from_numpy(spread_cum(R, B, V).astype(np.float32)).to(DEV)
        space = pa.alloc_workspace(pa.beam_select_workspace_size(R, B, V), DEV)
        out = tuple(torch.zeros((R, 6), dtype=d, device=DEV) for d in (torch.float32, torch.int32, torch.int32))
        want = [call(torch.roll(x, 17 * i, 1), cum, 6) for i in range(20)]
        jobs.append((x, cum, space, out, want, [[] for _ in out]))
    torch.cuda.synchronize()
    for i in range(20):
        for side, (x, cum, space, out, _, got) in zip(sides, jobs):
            with torch.cuda.stream(side):
                call(torch.roll(x, 17 * i, 1), cum, 6, space=space, out=out)
                for g, o in zip(got, out):
                    g.append(o.clone())
    torch.cuda.synchronize()
    for *_, want, got in jobs:
        for i in range(20):
            assert all(torch.equal(got[k][i], want[i][k]) for k in range(3))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,B,V", [(1, 4, 32000), (15, 3, 9001), (16, 3, 9001), (2, 32, 2048), (3, 1, 131072), (2, 5, 50001),
                                   (1, 31, 70), (4, 8, 128000)])
def test_captured_calls_give_the_same_bits(R, B, V, dtype):
    """A call outside a capture may take one launch for two; scores, beams and tokens stay the same."""
    x, cum = normal(R * B, V, R + V, dtype).to(DEV), torch.from_numpy(spread_cum(R, B, V).astype(np.float32)).to(DEV)
    want = check(x, cum.cpu().numpy(), 9)
    out = tuple(torch.zeros_like(t) for t in want)
    space = pa.alloc_workspace(pa.beam_select_workspace_size(R, B, V), DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, cum, 9, space=space, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    mine = tuple(torch.zeros_like(t) for t in want)
    call(x, cum, 9, space=space, out=mine, stream=torch.cuda.default_stream())
    assert all(torch.equal(a, b) for a, b in zip(mine, want))


def test_offsets_past_32_bits():
    """The last of many rows lies more than 2^31 elements behind the first."""
    R, B, V = 9, 32, 1 << 23
    stride = V + 8
    buffer = torch.empty(R * B * stride, dtype=torch.bfloat16, device=DEV)
    rows = buffer.as_strided((R * B, V), (stride, 1))
    cum = torch.full((R, B), -float("inf"), device=DEV)
    cum[R - 1, [3, B - 1]] = torch.tensor([-1.0, -1.5], device=DEV)
    x = normal(2, V, 71, torch.bfloat16)
    rows[(R - 1) * B + 3], rows[R * B - 1] = x[0].to(DEV), x[1].to(DEV)
    got = call(rows, cum, 6)
    sc, bm, tk, closest = ref.select(x.double().numpy(), np.array([[-1.0, -1.5]]), 6)
    assert closest > 2 * NEAR
    assert np.array_equal(got[1][R - 1].cpu().numpy(), np.array([3, B - 1])[bm[0]])
    assert np.array_equal(got[2][R - 1].cpu().numpy(), tk[0]) and (got[1][:R - 1] == -1).all()
