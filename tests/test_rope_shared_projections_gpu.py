"""pa_rope and pa_rope_append in place in projections whose q, k and v lie beside one another head by head
([tokens][heads][3][head_dim]): the results of calls into tensors of their own, which are compared with the
rotation in 64 bits (tests/rope_beam_ref.py), and nothing else in the projection changed."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa
from tests import rope_beam_ref as ref
from tests.test_rope_gpu import check_rows, pools, some_positions, values

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()
    yield
    assert pa.device_status() == 0


# pairs by eights, interleaved ones, any number of pairs; 3001 tokens are more than CTAs at a time
CASES = [(1, 2, 64, 64, False), (5, 3, 128, 128, False), (3001, 4, 64, 32, False), (7, 8, 256, 64, True),
         (3001, 3, 128, 38, True), (3001, 2, 64, 20, False), (4, 5, 128, 100, False)]


@pytest.mark.parametrize("first", ["tokens", "heads"])
@pytest.mark.parametrize("tokens,heads,hd,rotary,interleaved", CASES)
def test_rope(tokens, heads, hd, rotary, interleaved, first):
    x = values((tokens, heads, 3, hd) if first == "tokens" else (heads, tokens, 3, hd), 81).to(DEV)
    before = x.clone()
    q, k = ((x[..., i, :] if first == "tokens" else x[..., i, :].transpose(0, 1)) for i in (0, 1))
    pos = some_positions(tokens, 82)
    at = torch.from_numpy(pos).to(DEV)
    turns, _ = pa.rope_table(rotary)
    want_q, want_k = (torch.empty((tokens, heads, hd), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pa.pa_rope(want_q, want_k, q, k, at, turns, interleaved=interleaved)
    f, _ = ref.frequencies(rotary)
    check_rows(want_q, q, pos, f, 1.0, interleaved, what="q")
    check_rows(want_k, k, pos, f, 1.0, interleaved, what="k")
    pa.pa_rope(q, k, q, k, at, turns, interleaved=interleaved)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(x[..., 2, :], before[..., 2, :])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens,heads,hd,rotary,interleaved", CASES)
def test_append(tokens, heads, hd, rotary, interleaved, fp8):
    blocks = tokens // 16 + 2
    x = values((tokens, heads, 3, hd), 83).to(DEV)
    before = x.clone()
    at = torch.from_numpy(some_positions(tokens, 84)).to(DEV)
    slots = torch.from_numpy(np.random.default_rng(85).permutation(blocks * 16)[:tokens]).to(DEV)
    slots[tokens // 2] = -1                            # padding: its row stays
    turns, _ = pa.rope_table(rotary)
    own = pools(blocks, heads, hd, fp8, "HND", 86)
    mine = [c.clone() for c in own]
    q, k, v = (before[:, :, i].contiguous() for i in range(3))
    q_out = q.clone()
    pa.pa_rope_append(q_out, q, k, v, *own, slots, at, turns, interleaved=interleaved, k_scale=0.0137, v_scale=1 / 32)
    pa.pa_rope_append(x[:, :, 0], x[:, :, 0], x[:, :, 1], x[:, :, 2], *mine, slots, at, turns, interleaved=interleaved,
                      k_scale=0.0137, v_scale=1 / 32)
    assert torch.equal(x[:, :, 0], q_out) and torch.equal(x[:, :, 1:], before[:, :, 1:])
    assert torch.equal(x[tokens // 2], before[tokens // 2])
    for a, b in zip(mine, own):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
