"""Refusals of the rotary and beam-search entry points: by the library on the host (validation comes
before any CUDA call) and by the binding, whose operands the kernels would misread.  No GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_15_gb300 as pa
from tests import rope_beam_ref as ref


def at(i):
    """Buffers far from one another."""
    return 0x100000000 * (i + 1)


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return pa.load()


# ---- the table ----------------------------------------------------------------------------

@pytest.mark.parametrize("rotary", [2, 6, 64, 128, 256])
@pytest.mark.parametrize("scaling", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                     dict(scaling="bands", factor=8.0, original_len=8192),
                                     dict(scaling="bands", factor=2.5, original_len=100, low=0.5, high=7.0),
                                     dict(scaling="yarn", factor=32.0, original_len=4096),
                                     dict(scaling="yarn", factor=0.5, original_len=64, low=2.0, high=9.0)])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_table(rotary, scaling, base):
    if rotary == 2 and scaling.get("scaling") == "ntk":
        with pytest.raises(pa.PaError, match="no second frequency"):
            pa.rope_table(rotary, base, device="cpu", **scaling)
        return
    turns, m = pa.rope_table(rotary, base, device="cpu", **scaling)
    f, want_m = ref.frequencies(rotary, base, **scaling)
    assert turns.dtype == torch.int64 and turns.shape == (rotary // 2,)
    got = turns.numpy().astype(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    # a few roundings of 64-bit powers and logarithms; entries are whole units of 2^-64 of a turn, the
    # nearest one: off by half a unit, pi 2^-64 radians
    assert (np.abs(got - f) <= f * 2.0 ** -46 + math.pi * 2.0 ** -64).all() and abs(m - want_m) <= want_m * 2.0 ** -23


def test_table_of_any_frequencies():
    f = [1.0, 0.0, -1.0, 2 * math.pi * 3.25, 1e-12, -2 * math.pi * 5]
    t = pa.rope_table_of(f, device="cpu").numpy().astype(np.uint64)
    turns = t.astype(np.float64) / 2.0 ** 64
    want = np.remainder(np.array(f) / (2 * math.pi), 1.0)
    assert (np.abs(turns - want) <= 2.0 ** -50).all() and int(t[0]) + int(t[2]) == 1 << 64


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), 1), (dict(n=-2), 1), (dict(n=7), 1), (dict(n=258), 1), (dict(base=1.0), 1), (dict(base=0.0), 1),
    (dict(base=float("nan")), 1), (dict(base=float("inf")), 1), (dict(how=-1), 2), (dict(how=5), 2),
    (dict(how=1, s=0.0), 1), (dict(how=1, s=float("inf")), 1), (dict(how=2, s=-1.0), 1), (dict(how=2, n=2), 1),
    (dict(how=3, low=0.0), 1), (dict(how=3, low=4.0), 1), (dict(how=4, length=0), 1), (dict(how=3, length=-5), 1),
    (dict(how=4, high=float("inf")), 1), (dict(out=None), 1), (dict(), 0), (dict(how=2, s=2.0, n=4), 0),
])
def test_table_refusals(lib, kw, code):
    room = (ctypes.c_uint64 * 128)()
    a = dict(n=64, base=1e4, how=0, s=2.0, low=1.0, high=4.0, length=64, out=room)
    a.update(kw)
    assert lib.pa_rope_table(a["out"], None, a["n"], a["base"], a["how"], a["s"], a["low"], a["high"],
                             a["length"]) == code


def test_table_of_refusals(lib):
    room, f = (ctypes.c_uint64 * 4)(), (ctypes.c_double * 4)(1, 2, float("nan"), 4)
    assert lib.pa_rope_table_of(room, f, 2) == 0
    assert [lib.pa_rope_table_of(room, f, n) for n in (0, 3, 129, -1)] == [1] * 4
    assert lib.pa_rope_table_of(None, f, 2) == lib.pa_rope_table_of(room, None, 2) == 1
    with pytest.raises(ValueError, match="scaling"):
        pa.rope_table(64, scaling="su", device="cpu")
    with pytest.raises(pa.PaError):
        pa.rope_table(7, device="cpu")


# ---- the rotation -------------------------------------------------------------------------

S = 12 * 128      # a fused row: 8 query, 2 key, 2 value heads of 128 channels


def rope(lib, **kw):
    a = dict(qo=at(0), ko=at(1), q=at(2), k=at(3), pos=at(4), turns=at(5), T=4, nq=8, nk=2, hd=128, R=64, qot=1024,
             qoh=128, kot=256, koh=128, qt=1024, qh=128, kt=256, kh=128, m=1.0)
    a.update(kw)
    return lib.pa_rope(a["qo"], a["ko"], a["q"], a["k"], a["pos"], a["turns"], a["T"], a["nq"], a["nk"], a["hd"], a["R"],
                       a["qot"], a["qoh"], a["kot"], a["koh"], a["qt"], a["qh"], a["kt"], a["kh"], 0, 0, a["m"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(T=1 << 31), 2), (dict(nq=-1), 1), (dict(nk=70000), 2), (dict(hd=96), 2), (dict(R=0), 1),
    (dict(R=63), 1), (dict(R=130), 1), (dict(m=float("nan")), 1), (dict(m=float("inf")), 1), (dict(pos=None), 1),
    (dict(pos=at(4) + 4), 1), (dict(turns=at(5) + 4), 1),
    (dict(turns=None), 1), (dict(q=None), 1), (dict(qo=None), 1), (dict(k=at(3) + 8), 1), (dict(ko=at(1) + 2), 1),
    (dict(qt=1020), 1), (dict(kh=-128), 1), (dict(qt=1 << 60), 1), (dict(kot=0), 1), (dict(qoh=64), 1), (dict(qoh=0), 1),
    (dict(qot=512), 1),                                # a token's heads reach into the next token's
    (dict(qo=at(2) + 128), 1),                         # over q, but not in place
    (dict(qo=at(2), qot=2048), 1), (dict(ko=at(2)), 1), (dict(qo=at(3)), 1), (dict(qo=at(0), ko=at(0)), 1),
    (dict(ko=at(0) + 4 * 1024 * 2 - 16), 1),           # the outputs' ends meet
    # slices of one projection: k's result over a value slice of other rows is not seen to be apart
    (dict(q=at(2), qt=S, k=at(2) + 2048, kt=S, qo=at(2) + 256, qot=S), 1),
    (dict(T=0, q=None), 0), (dict(nq=0, nk=0), 0),
])
def test_rope_refusals(lib, kw, code):
    assert rope(lib, **kw) == code, lib.pa_last_error()


def append(lib, **kw):
    a = dict(qo=at(0), q=at(1), k=at(2), v=at(3), kc=at(4), vc=at(5), slots=at(6), pos=at(7), turns=at(8), T=4, nq=8,
             nkv=2, hd=128, R=64, bs=16, nb=10, qot=1024, qoh=128, qt=1024, qh=128, kt=256, kh=128, vt=256, vh=128,
             sb=4096, sh=2048, st=128, m=1.0, dt=0, ks=1.0, vs=1.0)
    a.update(kw)
    return lib.pa_rope_append(a["qo"], a["q"], a["k"], a["v"], a["kc"], a["vc"], a["slots"], a["pos"], a["turns"], a["T"],
                              a["nq"], a["nkv"], a["hd"], a["R"], a["bs"], a["nb"], a["qot"], a["qoh"], a["qt"], a["qh"],
                              a["kt"], a["kh"], a["vt"], a["vh"], a["sb"], a["sh"], a["st"], 0, a["m"], a["dt"], a["ks"],
                              a["vs"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(nq=-1), 1), (dict(nkv=0), 1), (dict(hd=80), 2), (dict(R=1), 1), (dict(bs=8), 2), (dict(nb=0), 1),
    (dict(st=64), 1), (dict(sh=0), 1), (dict(sb=4100), 1), (dict(dt=2), 2), (dict(dt=1, ks=0.0), 1),
    (dict(dt=1, vs=float("inf")), 1), (dict(dt=1, sb=4104), 1), (dict(slots=None), 1), (dict(kc=None), 1), (dict(vc=at(5) + 8), 1),
    (dict(q=None), 1), (dict(v=None), 1), (dict(k=at(2) + 4), 1), (dict(vt=100), 1), (dict(qo=at(1) + 16), 1),
    (dict(qo=at(2)), 1), (dict(qo=at(3)), 1), (dict(qot=256), 1), (dict(m=float("-inf")), 1), (dict(T=0), 0),
    (dict(pos=at(7) + 4), 1), (dict(turns=at(8) + 1), 1), (dict(slots=at(6) + 4), 1),
])
def test_append_refusals(lib, kw, code):
    assert append(lib, **kw) == code, lib.pa_last_error()


# ---- the beams ----------------------------------------------------------------------------

def select(lib, **kw):
    a = dict(sc=at(0), bm=at(1), tk=at(2), lg=at(3), cum=at(4), fin=None, end=0, R=2, B=4, V=1000, K=8, sr=1000, dt=0,
             ws=at(5), bytes=1 << 40)
    a.update(kw)
    return lib.pa_beam_select(a["sc"], a["bm"], a["tk"], a["lg"], a["cum"], a["fin"], a["end"], a["R"], a["B"], a["V"],
                              a["K"], a["sr"], a["dt"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), 1), (dict(B=0), 1), (dict(V=0), 1), (dict(K=0), 1), (dict(B=33), 2), (dict(K=65), 2),
    (dict(V=(1 << 24) + 1, sr=1 << 25), 2), (dict(dt=2), 2), (dict(dt=-1), 2), (dict(sr=999), 1), (dict(sr=-1), 1),
    (dict(sr=1 << 50), 2), (dict(fin=at(6), end=-1), 1), (dict(fin=at(6), end=1000), 1), (dict(sc=None), 1), (dict(bm=None), 1),
    (dict(tk=None), 1), (dict(lg=None), 1), (dict(cum=None), 1), (dict(lg=at(3) + 2), 1), (dict(lg=at(3) + 1, dt=1), 1),
    (dict(sc=at(0) + 2), 1), (dict(bm=at(1) + 1), 1), (dict(tk=at(2) + 3), 1), (dict(cum=at(4) + 2), 1),
    (dict(ws=None), 4), (dict(ws=at(5) + 16), 4), (dict(bytes=0), 4), (dict(sc=at(4)), 1), (dict(bm=at(4) + 28), 1),
    (dict(bm=at(0) + 60), 1), (dict(tk=at(1)), 1), (dict(sc=at(2)), 1), (dict(tk=at(3) + 7999 * 4), 1),
    (dict(sc=at(6), fin=at(6) + 7), 1), (dict(sc=at(6) - 60, fin=at(6)), 1), (dict(R=0), 0), (dict(R=0, sc=None), 0),
])
def test_select_refusals(lib, kw, code):
    assert select(lib, **kw) == code, lib.pa_last_error()


def test_select_refuses_a_workspace_one_byte_short(lib):
    need = pa.beam_select_workspace_size(2, 4, 1000)
    assert need >= 2 * 4 * 4 * 12 and need % 256 == 0
    assert select(lib, bytes=need - 1) == pa.PA_ERR_WORKSPACE
    assert [pa.beam_select_workspace_size(*x) for x in ((0, 4, 10), (2, -1, 10), (2, 4, 0))] == [0, 0, 0]


def reorder(lib, **kw):
    a = dict(pools=(ctypes.c_void_p * 2)(at(0), at(1)), n=2, bt=at(2), sl=at(3), of=at(4), R=2, B=4, nkv=2, hd=128, bs=16,
             mb=4, nb=10, sb=4096, sh=2048, st=128, dt=0)
    a.update(kw)
    return lib.pa_beam_reorder(a["pools"], a["n"], a["bt"], a["sl"], a["of"], a["R"], a["B"], a["nkv"], a["hd"], a["bs"],
                               a["mb"], a["nb"], a["sb"], a["sh"], a["st"], a["dt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 1), (dict(R=-1), 1), (dict(B=0), 1), (dict(B=33), 2), (dict(R=65536), 2), (dict(nkv=0), 1), (dict(nkv=65537), 2),
    (dict(hd=80), 2), (dict(bs=8), 2), (dict(nb=0), 1), (dict(mb=0), 1), (dict(mb=1 << 28), 1), (dict(st=64), 1), (dict(dt=2), 2),
    (dict(pools=None), 1), (dict(bt=None), 1), (dict(sl=None), 1), (dict(of=None), 1),
    (dict(pools=(ctypes.c_void_p * 2)(at(0), at(1) + 8)), 1), (dict(pools=(ctypes.c_void_p * 2)(at(0), 0)), 1),
    (dict(pools=(ctypes.c_void_p * 2)(at(0), at(0))), 1), (dict(sl=at(2) + 8 * 4 * 4 - 4), 1), (dict(of=at(2) - 28), 1),
    (dict(bt=at(2) + 2), 1), (dict(sl=at(3) + 1), 1), (dict(of=at(4) + 2), 1), (dict(R=0), 0), (dict(R=0, pools=None), 0),
])
def test_reorder_refusals(lib, kw, code):
    assert reorder(lib, **kw) == code, lib.pa_last_error()


# ---- the binding --------------------------------------------------------------------------

NB, NKV, HD, NQ, T, R, B, V = 6, 2, 64, 4, 3, 2, 3, 50


def rows(heads, t=T):
    return torch.zeros((t, heads, HD), dtype=torch.bfloat16)


def i64(n):
    return torch.zeros(n, dtype=torch.int64)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def pool(dtype=torch.bfloat16):
    return torch.zeros((NB, NKV, 16, HD), dtype=dtype)


def call_rope(**kw):
    a = dict(q_out=rows(NQ), k_out=rows(NKV), q=rows(NQ), k=rows(NKV), positions=i64(T), turns=i64(16))
    a.update(kw)
    pa.pa_rope(**a)


def call_append(**kw):
    a = dict(q_out=rows(NQ), q=rows(NQ), k=rows(NKV), v=rows(NKV), k_cache=pool(), v_cache=pool(), slot_mapping=i64(T),
             positions=i64(T), turns=i64(16))
    a.update(kw)
    pa.pa_rope_append(**a)


def call_select(**kw):
    a = dict(scores=torch.zeros((R, 4)), beams=i32(R, 4), tokens=i32(R, 4), logits=torch.zeros((R * B, V)),
             cum_scores=torch.zeros((R, B)), workspace=torch.zeros(1 << 16, dtype=torch.uint8),
             finished=torch.zeros((R, B), dtype=torch.bool))
    a.update(kw)
    pa.pa_beam_select(**a)


def call_reorder(**kw):
    a = dict(key_caches=[pool(), pool()], value_caches=[pool(), pool()], block_tables=i32(R * B, 4), seq_lens=i32(R * B),
             parents=i32(R, B))
    a.update(kw)
    pa.pa_beam_reorder(**a)


CALLS = {call_rope: 6, call_append: 9, call_select: 7, call_reorder: 7}


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors(call):
    with pytest.raises(AssertionError, match="current CUDA device"):
        call()


@pytest.mark.parametrize("call", CALLS)
def test_one_tensor_elsewhere_among_device_tensors(call, monkeypatch):
    """Every tensor of a call is looked at: all claim the current device but one at a time."""
    class Library:              # nothing is launched
        def __getattr__(self, name):
            return lambda *args: pa.PA_OK
    monkeypatch.setattr(pa, "load", Library)
    monkeypatch.setattr(pa, "_stream", lambda *args: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    seen = []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: seen.append(t) or 0)
    call()
    assert len({id(t) for t in seen}) == CALLS[call]
    n = len(seen)
    for bad in range(n):
        for elsewhere in (-1, 1):
            seen = []
            monkeypatch.setattr(torch.Tensor, "get_device",
                                lambda t: seen.append(t) or (elsewhere if len(seen) == bad + 1 else 0))
            with pytest.raises(AssertionError, match="current CUDA device"):
                call()


@pytest.mark.parametrize("call,kw,what", [
    (call_rope, dict(q=rows(NQ).float()), "bf16"), (call_rope, dict(k_out=rows(NKV).half()), "bf16"),
    (call_rope, dict(q_out=rows(NQ, T + 1)), "one token count"), (call_rope, dict(k=rows(NKV, T - 1)), "one token count"),
    (call_rope, dict(q_out=rows(NQ + 1)), "like q"), (call_rope, dict(k_out=rows(NKV + 1)), "like"),
    (call_rope, dict(k=None), "like"), (call_rope, dict(q=torch.zeros((T, NQ, 2 * HD), dtype=torch.bfloat16)[..., ::2]), "contiguous"),
    (call_rope, dict(positions=i32(T)), "int64"), (call_rope, dict(positions=i64(T + 1)), "int64"),
    (call_rope, dict(positions=i64(2 * T)[::2]), "int64"), (call_rope, dict(turns=torch.zeros(16)), "int64"),
    (call_append, dict(slot_mapping=i32(T)), "int64"), (call_append, dict(slot_mapping=i64(T - 1)), "int64"),
    (call_append, dict(k=rows(NKV + 1)), "heads"), (call_append, dict(v=rows(1)), "heads"), (call_append, dict(q=None), "heads"),
    (call_append, dict(v_cache=pool(torch.uint8)), "geometry"), (call_append, dict(v=rows(NKV).float()), "bf16"),
    (call_select, dict(logits=torch.zeros((R * B, V), dtype=torch.float16)), "logits"),
    (call_select, dict(logits=torch.zeros((R * B + 1, V))), "logits"), (call_select, dict(logits=torch.zeros((V, R * B)).T), "logits"),
    (call_select, dict(cum_scores=torch.zeros((R, B), dtype=torch.float64)), "float32"),
    (call_select, dict(cum_scores=torch.zeros((B, R)).T), "float32"), (call_select, dict(scores=torch.zeros((R + 1, 4))), "scores"),
    (call_select, dict(beams=i32(R, 5)), "scores"), (call_select, dict(tokens=torch.zeros((R, 4), dtype=torch.int64)), "int32"),
    (call_select, dict(finished=torch.zeros((R, B))), "finished"), (call_select, dict(finished=torch.zeros((B, R), dtype=torch.bool)), "finished"),
    (call_reorder, dict(block_tables=i32(R * B + 1, 4)), "row per request"), (call_reorder, dict(parents=i64(R * B).view(R, B)), "int32"),
    (call_reorder, dict(block_tables=i32(R * B, 8)[:, ::2]), "int32"), (call_reorder, dict(seq_lens=i32(R * B - 1)), "int32"),
    (call_reorder, dict(value_caches=[pool(), pool()[:-1]]), "geometry"), (call_reorder, dict(value_caches=[pool()]), "key and a value pool"),
])
def test_operands(call, kw, what):
    with pytest.raises(AssertionError, match=what):
        call(**kw)
