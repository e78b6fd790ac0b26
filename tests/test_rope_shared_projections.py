"""Which results of pa_rope and pa_rope_append may stand in place in a projection that holds more than
one tensor, and which overlap another.  Host checks alone, on addresses that nothing is at: where there
is a device the accepted calls would be launched, so these run only where there is none (the same calls
on real tensors are in test_rope_shared_projections_gpu.py)."""
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa
from tests.test_rope_beam_refusals import append, at, lib, rope  # noqa: F401  (lib: a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

ACCEPTED = pa.PA_ERR_CUDA          # past every check, at the launch: no device
HD, H = 128, 8


def rows(base, token, head, name):
    """Arguments of a tensor and its result, in place."""
    out = {"q": ("qo", "qot", "qoh"), "k": ("ko", "kot", "koh")}[name]
    return {name: base, name + "t": token, name + "h": head, out[0]: base, out[1]: token, out[2]: head}


def both(q, k, token, head, k_token=None, k_head=None, **kw):
    return dict(rows(q, token, head, "q"), **rows(k, k_token or token, k_head or head, "k"), nq=H, nk=H, hd=HD, R=HD, **kw)


X = at(2)
PER_HEAD = 3 * HD                  # [tokens][heads][3][head_dim]
TOKEN = H * PER_HEAD


@pytest.mark.parametrize("what,kw,code", [
    ("q, k and v of a head beside one another", both(X, X + 2 * HD, TOKEN, PER_HEAD), ACCEPTED),
    ("k before q", both(X + 4 * HD, X, TOKEN, PER_HEAD), ACCEPTED),
    ("heads before tokens", both(X, X + 2 * HD, PER_HEAD, 4 * PER_HEAD), ACCEPTED),
    ("rows with a gap behind them", both(X, X + 2 * HD, TOKEN + PER_HEAD, PER_HEAD), ACCEPTED),
    ("one token", both(X, X + 2 * HD, 8, PER_HEAD, T=1), ACCEPTED),
    ("fewer k heads, each beside a q head", dict(both(X, X + 2 * HD, TOKEN, PER_HEAD), nk=3), ACCEPTED),
    ("k's heads twice as far apart", both(X, X + 2 * HD, 2 * TOKEN, PER_HEAD, k_head=2 * PER_HEAD), ACCEPTED),
    ("[tokens][2][heads][head_dim]", both(X, X + 2 * H * HD, 2 * H * HD, HD), ACCEPTED),
    ("k starts within q's head", both(X, X + 2 * (HD - 8), TOKEN, PER_HEAD), 1),
    ("k ends within the next head's q", both(X, X + 2 * (2 * HD + 8), TOKEN, PER_HEAD), 1),
    ("k starts within a later head", both(X, X + 2 * (2 * PER_HEAD + 64), TOKEN, PER_HEAD), 1),
    ("k ends within an earlier token's head", both(X + 2 * TOKEN, X + 2 * HD - 16, TOKEN, PER_HEAD), 1),
    ("heads that lie ever later in their period", both(X, X + 2 * HD, TOKEN, PER_HEAD, k_head=PER_HEAD + 8), 1),
    ("tokens that are no whole periods apart", both(X, X + 2 * HD, TOKEN, PER_HEAD, k_token=TOKEN + 64), 1),
])
def test_in_place(lib, what, kw, code):  # noqa: F811
    assert rope(lib, **kw) == code, lib.pa_last_error()


@pytest.mark.parametrize("what,kw,code", [
    ("q, k and v of a head beside one another", dict(), ACCEPTED),
    ("v first", dict(q=X + 2 * HD, qo=X + 2 * HD, k=X + 4 * HD, v=X), ACCEPTED),
    ("k starts within q's head", dict(k=X + 2 * (HD - 8)), 1),
    ("v ends within the next head's q", dict(v=X + 2 * (2 * HD + 8)), 1),
    ("q's result over v", dict(qo=X + 4 * HD), 1),
    ("q's result half over k", dict(qo=X + HD), 1),
])
def test_append(lib, what, kw, code):  # noqa: F811
    a = dict(qo=X, q=X, k=X + 2 * HD, v=X + 4 * HD, qot=TOKEN, qoh=PER_HEAD, qt=TOKEN, qh=PER_HEAD, kt=TOKEN, kh=PER_HEAD,
             vt=TOKEN, vh=PER_HEAD, nq=H, nkv=H, hd=HD, R=HD, sb=16 * H * HD, sh=16 * HD, st=HD)
    a.update(kw)
    assert append(lib, **a) == code, lib.pa_last_error()


def test_exhaustive_over_small_layouts(lib):  # noqa: F811
    """Accepted calls share no channel, by listing every one of them; and where the strides are whole periods of a
    common one, those that share none are accepted."""
    hd = 64
    refused_apart = 0
    for tokens, nq, nk in ((1, 2, 2), (2, 2, 2), (3, 2, 1), (2, 1, 3)):
        for qt, qh in ((192, 64), (256, 128), (128, 256), (384, 192), (512, 128), (200, 72)):
            for kt, kh in ((qt, qh), (qt, 2 * qh), (2 * qt, qh)):
                def channels(base, heads, st, sh):
                    return {base + t * st + h * sh + c for t in range(tokens) for h in range(heads) for c in range(0, hd, 8)}
                q = channels(0, nq, qt, qh)
                if len(q) < tokens * nq * hd // 8 or len(channels(0, nk, kt, kh)) < tokens * nk * hd // 8:
                    continue
                for d in range(-640, 648, 8):
                    k = channels(d, nk, kt, kh)
                    code = rope(lib, T=tokens, nq=nq, nk=nk, hd=hd, R=hd, q=X, qo=X, qt=qt, qot=qt, qh=qh, qoh=qh,
                                k=X + 2 * d, ko=X + 2 * d, kt=kt, kot=kt, kh=kh, koh=kh)
                    assert code in (1, ACCEPTED)
                    if code == ACCEPTED:
                        assert not q & k, (tokens, nq, nk, qt, qh, kt, kh, d)
                    refused_apart += code == 1 and not q & k and qt == kt and qh == kh and max(qt, qh) % min(qt, qh) == 0 \
                        and d % min(qt, qh) >= hd and d % min(qt, qh) + hd <= min(qt, qh)
    assert refused_apart == 0
