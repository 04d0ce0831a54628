"""Host-side argument checks of the calls for 4-bit caches, beams and pages (no GPU needed).
Every call here fails validation, or has nothing to do, before a device pointer is used."""
import ctypes

import pytest
import torch

import varlen_gated_delta_gb300 as gdn
from varlen_gated_delta_gb300 import build as gdn_build

P = ctypes.c_void_p(4096)
Q = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p(4100)


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load_library()


def _call(f, base, kw):
    return f(*dict(base, **kw).values())


WRITE = dict(k=P, v=P, ks=256, vs=256, slots=P, kscale=None, vscale=None, kc=P, vc=P, ko=None, vo=None, N=4, HKV=2, D=128, ps=16,
             pages=3, dtype=1, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 2), (dict(HKV=0), 2), (dict(D=0), 2), (dict(D=272), 2), (dict(D=120), 5), (dict(ps=0), 2), (dict(ps=24), 5),
    (dict(pages=0), 2), (dict(pages=1 << 28), 3), (dict(dtype=2), 5), (dict(ks=255), 2), (dict(vs=0), 2), (dict(vs=1 << 45), 3),
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(ko=P), 1),
    (dict(vo=P), 1), (dict(kc=ODD), 5), (dict(ko=ODD, vo=P), 5), (dict(N=0), 0)])
def test_kv4_write_refusals(lib, kw, status):
    assert _call(lib.gdn_kv4_write, WRITE, kw) == status
    assert status == 0 or lib.gdn_last_error()


ATTN = dict(q=P, kc=P, vc=P, kscale=None, vscale=None, table=P, kv=P, offsets=P, out=P, B=2, N=8, H=4, HKV=2, D=64, ps=16, M=4,
            pages=9, max_q=4, qs=256, scale=0.0, dtype=1, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 2), (dict(N=-1), 2), (dict(H=3), 2), (dict(H=0), 2), (dict(D=300), 2), (dict(D=72), 5), (dict(ps=0), 2), (dict(ps=8), 5),
    (dict(M=0), 2), (dict(pages=0), 2), (dict(max_q=-1), 2), (dict(pages=1 << 28), 3), (dict(M=1 << 28), 3), (dict(qs=100), 2),
    (dict(dtype=9), 5), (dict(scale=float("nan")), 2), (dict(q=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(table=None), 1),
    (dict(kv=None), 1), (dict(offsets=None), 1), (dict(out=None), 1), (dict(out=ODD), 5), (dict(vc=ODD), 5), (dict(ws=None), 8),
    (dict(ws=ODD), 8), (dict(ws_bytes=16), 8), (dict(N=0), 0), (dict(max_q=0), 0)])
def test_kv4_attention_refusals(lib, kw, status):
    assert _call(lib.gdn_attention_paged_kv4, ATTN, kw) == status


BEAM = dict(x=P, stride=1000, scores=P, done=None, end=-1, keep=0, tokens=P, parents=P, so=Q, fo=None, G=2, K=4, V=1000, n=4, dtype=1,
            ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(G=0), 2), (dict(K=0), 2), (dict(V=0), 2), (dict(n=0), 2), (dict(K=129), 5), (dict(n=129), 5), (dict(V=1, n=5), 2),
    (dict(V=1 << 30, stride=1 << 30), 3), (dict(G=1 << 28), 3), (dict(dtype=2), 5), (dict(stride=999), 2), (dict(stride=1 << 45), 3),
    (dict(keep=1, n=3), 2), (dict(done=P), 2), (dict(fo=P), 2), (dict(done=P, end=1000), 2), (dict(x=None), 1), (dict(scores=None), 1),
    (dict(tokens=None), 1), (dict(parents=None), 1), (dict(so=None), 1), (dict(so=P, n=5), 2), (dict(so=ODD), 2),
    (dict(done=P, fo=P, end=1, n=3), 2), (dict(ws=None), 8), (dict(ws=ODD), 8), (dict(ws_bytes=16), 8)])
def test_beam_select_refusals(lib, kw, status):
    assert _call(lib.gdn_beam_select, BEAM, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), 2), (dict(B=0), 2), (dict(count=65), 5), (dict(B=4097), 5), (dict(parents=None), 1), (dict(sizes=[-1, 8]), 2),
    (dict(sizes=[1 << 41, 8]), 3), (dict(ptrs=[0, 4096]), 1), (dict(ptrs=[4096, 4096]), 2), (dict(ptrs=[4096, 4100]), 2),
    (dict(ptrs=[4196, 4096], sizes=[8, 64]), 2), (dict(count=0), 0)])
def test_state_reorder_refusals(lib, kw, status):
    a = dict(dict(ptrs=[4096, 1 << 20], sizes=[64, 64], count=2, parents=P, B=2), **kw)
    ptrs, sizes = (ctypes.c_void_p * 2)(*a["ptrs"]), (ctypes.c_int64 * 2)(*a["sizes"])
    assert lib.gdn_state_reorder(ptrs, sizes, a["count"], a["parents"], a["B"], None) == status


FORK = dict(parents=P, kv=P, table=P, free=P, cursor=P, to=Q, ko=Q, copies=P, co=P, status=P, B=2, R=2, ps=16, M=4, pages=9, n_free=9,
            ws=P, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 2), (dict(R=0), 2), (dict(B=8193), 5), (dict(R=8193), 5), (dict(ps=0), 2), (dict(ps=65537), 2), (dict(M=0), 2),
    (dict(pages=0), 2), (dict(n_free=-1), 2), (dict(M=1 << 30), 3), (dict(parents=None), 1), (dict(kv=None), 1), (dict(table=None), 1),
    (dict(free=None), 1), (dict(cursor=None), 1), (dict(to=None), 1), (dict(ko=None), 1), (dict(copies=None), 1), (dict(co=None), 1),
    (dict(status=None), 1), (dict(copies=ODD), 5), (dict(to=P, R=3), 2), (dict(ko=P, R=3), 2), (dict(to=ODD), 2), (dict(ko=ODD), 2),
    (dict(ws=None), 8), (dict(ws=ODD), 8), (dict(ws_bytes=16), 8)])
def test_page_fork_refusals(lib, kw, status):
    assert _call(lib.gdn_page_fork, FORK, kw) == status


COMPACT = dict(kv=P, table=P, to=Q, copies=P, free=P, co=P, status=P, B=2, ps=16, M=4, pages=9, ws=P, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 2), (dict(ps=0), 2), (dict(M=0), 2), (dict(pages=0), 2), (dict(M=1 << 30), 3), (dict(kv=None), 1), (dict(table=None), 1),
    (dict(to=None), 1), (dict(copies=None), 1), (dict(free=None), 1), (dict(co=None), 1), (dict(status=None), 1), (dict(copies=ODD), 5),
    (dict(to=ODD), 2), (dict(ws=None), 8), (dict(ws=ODD), 8), (dict(ws_bytes=16), 8)])
def test_page_compact_refusals(lib, kw, status):
    assert _call(lib.gdn_page_compact, COMPACT, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), 2), (dict(n=-1), 2), (dict(pages=-1), 2), (dict(count=129), 5), (dict(copies=None), 1), (dict(copies=ODD), 5),
    (dict(sizes=[-1, 8]), 2), (dict(sizes=[1 << 33, 8]), 3), (dict(ptrs=[0, 4096]), 1), (dict(count=0), 0), (dict(n=0), 0),
    (dict(pages=0), 0)])
def test_page_copy_refusals(lib, kw, status):
    a = dict(dict(ptrs=[4096, 1 << 20], sizes=[64, 64], count=2, copies=P, n=3, pages=5), **kw)
    ptrs, sizes = (ctypes.c_void_p * 2)(*a["ptrs"]), (ctypes.c_int64 * 2)(*a["sizes"])
    assert lib.gdn_page_copy(ptrs, sizes, a["count"], a["copies"], a["n"], a["pages"], None) == status


@pytest.mark.parametrize("D", [16, 256])
def test_kv4_pages_past_32_bit_places_are_refused(lib, D):
    for ps, status in ((1 << 20, 0), ((1 << 20) + 16, 3), (1 << 24, 3)):
        assert _call(lib.gdn_kv4_write, WRITE, dict(ps=ps, pages=1, D=D, ks=512, vs=512, N=0)) == status
        assert _call(lib.gdn_attention_paged_kv4, ATTN, dict(ps=ps, pages=1, M=1, D=D, qs=1024, N=0)) == status


def test_workspace_queries(lib):
    attn, beam = gdn.gdn_attention_paged_kv4_workspace_bytes, gdn.gdn_beam_select_workspace_bytes
    assert attn(64, 64, 32, 8, 128, 1) > 0
    assert attn(0, 64, 32, 8, 128, 1) == attn(4, 4, 3, 2, 64, 1) == attn(4, 4, 4, 2, 72, 1) == attn(4, -1, 4, 2, 64, 1) == 0
    assert beam(1, 4, 32768, 4) > 0 and beam(0, 4, 32768, 4) == beam(1, 129, 10, 4) == beam(1, 1, 3, 4) == 0
    assert gdn.gdn_page_fork_workspace_bytes(2, 4, 9) > 0 and gdn.gdn_page_fork_workspace_bytes(0, 4, 9) == 0
    assert gdn.gdn_page_compact_workspace_bytes(9) > 0 and gdn.gdn_page_compact_workspace_bytes(0) == 0
    assert gdn.kv4_page_bytes(64, 128) == 64 * 72


@pytest.mark.parametrize("call", [
    lambda t: gdn.gdn_kv4_write(t, t, t, t, t), lambda t: gdn.gdn_beam_select(t, t), lambda t: gdn.gdn_state_reorder([t], t),
    lambda t: gdn.gdn_page_fork(t, t, t, t, page_size=16, num_pages=4, cursor=t),
    lambda t: gdn.gdn_page_compact(t, t, page_size=16, num_pages=4), lambda t: gdn.gdn_page_copy([t], t),
    lambda t: gdn.gdn_attention_paged_kv4(t, t, t, t, t, t, max_q=1)])
def test_python_calls_refuse_host_tensors(lib, call):
    with pytest.raises(gdn.GdnError):
        call(torch.zeros(2, 2))
    with pytest.raises(TypeError):
        call(3)
