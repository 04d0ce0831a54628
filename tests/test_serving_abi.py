"""Host-side argument checks of the softmax-attention serving calls (no GPU needed).
Every call here fails validation, or has nothing to do, before a pointer is used."""
import ctypes

import pytest

import varlen_gated_delta_gb300 as gdn
from varlen_gated_delta_gb300 import build as gdn_build

P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load_library()


def _plan(lib, **kw):
    a = dict(new=P, cached=P, table=P, free=P, cursor=P, offsets=P, kv=P, pos=P, slots=P, cout=P, status=P, B=2, N=8,
             ps=16, M=4, n_free=10, stream=None)
    a.update(kw)
    return lib.gdn_page_plan(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 2), (dict(N=-1), 2), (dict(ps=0), 2), (dict(ps=65537), 2), (dict(M=0), 2), (dict(n_free=-1), 2),
    (dict(B=8193), 5), (dict(new=None), 1), (dict(cached=None), 1), (dict(table=None), 1), (dict(free=None), 1),
    (dict(cursor=None), 1), (dict(offsets=None), 1), (dict(kv=None), 1), (dict(pos=None), 1), (dict(slots=None), 1),
    (dict(cout=None), 1), (dict(status=None), 1)])
def test_page_plan_refusals(lib, kw, status):
    assert _plan(lib, **kw) == status
    assert lib.gdn_last_error()


def _rope(lib, **kw):
    a = dict(qkv=P, stride=1024, qw=P, kw=P, eps=1e-6, cs=P, pos=P, max_pos=10, slots=P, q=P, k=P, kc=P, vc=P, num_slots=8,
             N=4, H=4, HKV=2, D=128, R=128, style=0, dtype=1, stream=None)
    a.update(kw)
    return lib.gdn_qk_norm_rope(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 2), (dict(H=0), 2), (dict(HKV=3), 2), (dict(D=257), 2), (dict(D=0), 2), (dict(R=3), 2), (dict(R=130), 2),
    (dict(R=-2), 2), (dict(style=2), 5), (dict(dtype=3), 5), (dict(stride=1023), 2), (dict(stride=1 << 45), 3),
    (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(max_pos=0), 2), (dict(num_slots=-1), 2), (dict(qkv=None), 1),
    (dict(q=None), 1), (dict(cs=None), 1), (dict(pos=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(N=0), 0)])
def test_qk_norm_rope_refusals(lib, kw, status):
    assert _rope(lib, **kw) == status


def _varlen(lib, **kw):
    a = dict(q=P, k=P, v=P, offsets=P, out=P, B=2, N=8, H=4, HKV=2, D=64, qs=256, ks=128, vs=128, scale=0.0, dtype=1,
             stream=None)
    a.update(kw)
    return lib.gdn_attention_varlen(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 2), (dict(N=-1), 2), (dict(H=3), 2), (dict(HKV=0), 2), (dict(D=300), 2), (dict(qs=255), 2), (dict(ks=127), 2),
    (dict(vs=0), 2), (dict(vs=-128), 2), (dict(qs=1 << 50), 3), (dict(dtype=2), 5), (dict(scale=float("inf")), 2),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(offsets=None), 1), (dict(out=None), 1), (dict(N=0), 0)])
def test_attention_varlen_refusals(lib, kw, status):
    assert _varlen(lib, **kw) == status


def _paged(lib, **kw):
    a = dict(q=P, k=P, v=P, table=P, kv=P, offsets=P, out=P, B=2, N=8, H=4, HKV=2, D=64, ps=16, M=4, pages=9, max_q=4, qs=256,
             scale=0.0, dtype=1, ws=P, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.gdn_attention_paged(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 2), (dict(N=-1), 2), (dict(H=3), 2), (dict(D=300), 2), (dict(ps=0), 2), (dict(M=0), 2), (dict(pages=0), 2),
    (dict(max_q=-1), 2), (dict(pages=1 << 28), 3), (dict(M=1 << 28), 3), (dict(qs=100), 2), (dict(dtype=9), 5),
    (dict(scale=float("nan")), 2), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(table=None), 1),
    (dict(kv=None), 1), (dict(offsets=None), 1), (dict(out=None), 1), (dict(ws=None), 8), (dict(ws=ctypes.c_void_p(4100)), 8),
    (dict(ws_bytes=16), 8), (dict(N=0), 0), (dict(max_q=0), 0)])
def test_attention_paged_refusals(lib, kw, status):
    assert _paged(lib, **kw) == status


def test_paged_workspace_query():
    size = gdn.gdn_attention_paged_workspace_bytes
    assert size(64, 64, 32, 8, 128, 1) > 0
    assert size(0, 64, 32, 8, 128, 1) == size(4, 4, 3, 2, 64, 1) == size(4, 4, 4, 2, 300, 1) == size(4, -1, 4, 2, 64, 1) == 0
