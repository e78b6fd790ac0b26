"""Host-side refusals of the tree and page-selection entry points (no GPU: validation comes
before any CUDA call)."""
import ctypes

import pytest

import paged_kv_gqa_15_gb300 as pa

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
OFF4 = ctypes.c_void_p(0x10004)
OFF16 = ctypes.c_void_p(0x10010)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return pa.load()


def tree(lib, **kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, ip=FAKE, mask=FAKE, words=1, B=2, rows=8,
             T=8, nq=8, nkv=2, hd=128, bs=16, mb=4, nb=100, sb=4096, sh=2048, st=128, scale=0.1, win=0, dt=0,
             ks=1.0, vs=1.0, ws=FAKE, bytes=1 << 40)
    a.update(kw)
    return lib.pa_tree_decode(a["out"], a["q"], a["k"], a["v"], a["bt"], a["sl"], a["ip"], a["mask"], a["words"],
                              a["B"], a["rows"], a["T"], a["nq"], a["nkv"], a["hd"], a["bs"], a["mb"], a["nb"],
                              a["sb"], a["sh"], a["st"], a["scale"], a["win"], a["dt"], a["ks"], a["vs"], a["ws"],
                              a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(hd=96), pa.PA_ERR_UNSUPPORTED),
    (dict(nq=6, nkv=4), pa.PA_ERR_INVALID),
    (dict(nkv=0), pa.PA_ERR_INVALID),
    (dict(bs=32), pa.PA_ERR_UNSUPPORTED),
    (dict(nb=0), pa.PA_ERR_INVALID),
    (dict(nb=1 << 31), pa.PA_ERR_UNSUPPORTED),
    (dict(mb=0), pa.PA_ERR_INVALID),
    (dict(mb=1 << 28), pa.PA_ERR_INVALID),
    (dict(B=-1), pa.PA_ERR_INVALID),
    (dict(rows=-1), pa.PA_ERR_INVALID),
    (dict(T=-1), pa.PA_ERR_INVALID),
    (dict(T=257, words=5), pa.PA_ERR_UNSUPPORTED),
    (dict(T=65), pa.PA_ERR_INVALID),                  # two words are needed
    (dict(words=0), pa.PA_ERR_INVALID),
    (dict(scale=0.0), pa.PA_ERR_INVALID),
    (dict(scale=float("nan")), pa.PA_ERR_INVALID),
    (dict(scale=float("inf")), pa.PA_ERR_INVALID),
    (dict(scale=-1.0), pa.PA_ERR_INVALID),
    (dict(dt=3), pa.PA_ERR_UNSUPPORTED),
    (dict(dt=1, ks=0.0), pa.PA_ERR_INVALID),
    (dict(st=100), pa.PA_ERR_INVALID),
    (dict(st=64), pa.PA_ERR_INVALID),
    (dict(q=None), pa.PA_ERR_INVALID),
    (dict(mask=None), pa.PA_ERR_INVALID),
    (dict(ip=None), pa.PA_ERR_INVALID),
    (dict(out=ODD), pa.PA_ERR_INVALID),
    (dict(v=ODD), pa.PA_ERR_INVALID),
    (dict(mask=OFF4), pa.PA_ERR_INVALID),
    (dict(bytes=0), pa.PA_ERR_WORKSPACE),
    (dict(ws=None), pa.PA_ERR_WORKSPACE),
    (dict(ws=OFF16), pa.PA_ERR_WORKSPACE),
    (dict(B=0), pa.PA_OK),
    (dict(rows=0), pa.PA_OK),
    (dict(T=0, words=0), pa.PA_OK),
])
def test_tree_refusals(lib, kw, code):
    assert tree(lib, **kw) == code


def test_tree_refuses_a_workspace_one_byte_short(lib):
    need = pa.tree_decode_workspace_size(2, 8, 8, 2, 128)
    assert need > 0
    assert tree(lib, bytes=need - 1) == pa.PA_ERR_WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), pa.PA_ERR_INVALID),
    (dict(B=-1), pa.PA_ERR_INVALID),
    (dict(B=70000), pa.PA_ERR_UNSUPPORTED),
    (dict(hd=80), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=8), pa.PA_ERR_UNSUPPORTED),
    (dict(sh=0), pa.PA_ERR_INVALID),
    (dict(dt=2), pa.PA_ERR_UNSUPPORTED),
    (dict(T=-1), pa.PA_ERR_INVALID),
    (dict(A=-1), pa.PA_ERR_INVALID),
    (dict(mb=0), pa.PA_ERR_INVALID),
    (dict(acc=None), pa.PA_ERR_INVALID),
    (dict(pools=None), pa.PA_ERR_INVALID),
    (dict(new=FAKE), pa.PA_ERR_INVALID),              # seq_lens itself
    (dict(new=None), pa.PA_ERR_INVALID),
    (dict(pools=(ctypes.c_void_p * 2)(0x10000, 0x20008)), pa.PA_ERR_INVALID),
    (dict(pools=(ctypes.c_void_p * 2)(0x10000, 0)), pa.PA_ERR_INVALID),
    (dict(pools=(ctypes.c_void_p * 2)(0x10000, 0x10000)), pa.PA_ERR_INVALID),         # moved twice
    (dict(pools=(ctypes.c_void_p * 4)(0x10000, 0x20000, 0x30000, 0x20000), n=4), pa.PA_ERR_INVALID),
    (dict(new=OFF16, al=OFF16), pa.PA_ERR_INVALID),
    (dict(new=OFF4), pa.PA_ERR_INVALID),                                               # overlaps seq_lens
    (dict(B=0), pa.PA_OK),
])
def test_commit_refusals(lib, kw, code):
    a = dict(pools=(ctypes.c_void_p * 2)(0x10000, 0x20000), n=2, bt=FAKE, sl=FAKE, ip=FAKE, acc=FAKE, al=FAKE,
             new=OFF16, B=2, T=8, A=4, nkv=2, hd=128, bs=16, mb=4, nb=10, sb=4096, sh=2048, st=128, dt=0)
    a.update(kw)
    assert lib.pa_tree_commit(a["pools"], a["n"], a["bt"], a["sl"], a["ip"], a["acc"], a["al"], a["new"], a["B"],
                              a["T"], a["A"], a["nkv"], a["hd"], a["bs"], a["mb"], a["nb"], a["sb"], a["sh"],
                              a["st"], a["dt"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), pa.PA_ERR_INVALID),
    (dict(new=-1), pa.PA_ERR_INVALID),
    (dict(hd=80), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=8), pa.PA_ERR_UNSUPPORTED),
    (dict(nkv=0), pa.PA_ERR_INVALID),
    (dict(mb=0), pa.PA_ERR_INVALID),
    (dict(dt=2), pa.PA_ERR_UNSUPPORTED),
    (dict(bounds=None), pa.PA_ERR_INVALID),
    (dict(bounds=ODD), pa.PA_ERR_INVALID),
    (dict(k=ODD), pa.PA_ERR_INVALID),
    (dict(B=1 << 20, mb=1 << 20, new=1 << 24, nkv=8), pa.PA_ERR_UNSUPPORTED),
    (dict(B=0), pa.PA_OK),
    (dict(new=0), pa.PA_OK),
])
def test_bounds_refusals(lib, kw, code):
    a = dict(bounds=FAKE, k=FAKE, bt=FAKE, sl=FAKE, ft=None, new=8, B=2, nkv=2, hd=128, bs=16, mb=4, nb=10,
             sb=4096, sh=2048, st=128, dt=0)
    a.update(kw)
    assert lib.pa_page_bounds(a["bounds"], a["k"], a["bt"], a["sl"], a["ft"], a["new"], a["B"], a["nkv"], a["hd"],
                              a["bs"], a["mb"], a["nb"], a["sb"], a["sh"], a["st"], a["dt"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), pa.PA_ERR_INVALID),
    (dict(B=70000), pa.PA_ERR_UNSUPPORTED),
    (dict(nq=7), pa.PA_ERR_INVALID),
    (dict(hd=96), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=32), pa.PA_ERR_UNSUPPORTED),
    (dict(nb=0), pa.PA_ERR_INVALID),
    (dict(mb=0), pa.PA_ERR_INVALID),
    (dict(nb=1 << 27), pa.PA_ERR_UNSUPPORTED),
    (dict(mb=524289), pa.PA_ERR_UNSUPPORTED),
    (dict(most=0), pa.PA_ERR_INVALID),
    (dict(most=1 << 28), pa.PA_ERR_INVALID),
    (dict(sink=-1), pa.PA_ERR_INVALID),
    (dict(recent=0), pa.PA_ERR_INVALID),
    (dict(sink=3, recent=2), pa.PA_ERR_INVALID),
    (dict(sink=2147483647, recent=2147483647), pa.PA_ERR_INVALID),
    (dict(dt=5), pa.PA_ERR_UNSUPPORTED),
    (dict(q=None), pa.PA_ERR_INVALID),
    (dict(q=ODD), pa.PA_ERR_INVALID),
    (dict(bounds=ODD), pa.PA_ERR_INVALID),
    (dict(bytes=0), pa.PA_ERR_WORKSPACE),
    (dict(ws=OFF16), pa.PA_ERR_WORKSPACE),
    (dict(ws=None), pa.PA_ERR_WORKSPACE),
    (dict(pt=ODD), pa.PA_ERR_INVALID),                # over block_tables
    (dict(pt=ctypes.c_void_p(0x90000)), pa.PA_ERR_INVALID),   # page_lens is seq_lens
    (dict(B=0), pa.PA_OK),
])
def test_select_refusals(lib, kw, code):
    a = dict(pt=FAKE, pl=FAKE, q=FAKE, bounds=FAKE, bt=FAKE, sl=FAKE, B=2, nq=8, nkv=2, hd=128, bs=16, mb=8, nb=10,
             most=4, sink=1, recent=1, dt=0, ws=FAKE, bytes=1 << 40)
    a.update(kw)
    assert lib.pa_select_pages(a["pt"], a["pl"], a["q"], a["bounds"], a["bt"], a["sl"], a["B"], a["nq"], a["nkv"],
                               a["hd"], a["bs"], a["mb"], a["nb"], a["most"], a["sink"], a["recent"], a["dt"],
                               a["ws"], a["bytes"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(hd=96), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=32), pa.PA_ERR_UNSUPPORTED),
    (dict(mp=0), pa.PA_ERR_INVALID),
    (dict(mp=1 << 28), pa.PA_ERR_UNSUPPORTED),
    (dict(out=ODD), pa.PA_ERR_INVALID),
    (dict(pt=None), pa.PA_ERR_INVALID),
    (dict(bytes=0), pa.PA_ERR_WORKSPACE),
    (dict(ws=OFF16), pa.PA_ERR_WORKSPACE),
    (dict(dt=1, ks=-1.0), pa.PA_ERR_INVALID),
    (dict(B=0), pa.PA_OK),
])
def test_decode_pages_refusals(lib, kw, code):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, pt=FAKE, pl=FAKE, B=2, nq=8, nkv=2, hd=128, bs=16, mp=4, nb=10,
             sb=4096, sh=2048, st=128, scale=0.1, dt=0, ks=1.0, vs=1.0, ws=FAKE, bytes=1 << 40)
    a.update(kw)
    assert lib.pa_decode_pages(a["out"], a["q"], a["k"], a["v"], a["pt"], a["pl"], a["B"], a["nq"], a["nkv"],
                               a["hd"], a["bs"], a["mp"], a["nb"], a["sb"], a["sh"], a["st"], a["scale"], a["dt"],
                               a["ks"], a["vs"], a["ws"], a["bytes"], None) == code
