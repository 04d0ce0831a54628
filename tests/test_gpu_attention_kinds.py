"""Infinities and NaN in the values: which outputs become +inf, -inf or NaN is the same wherever the key lies in
a tile.  An infinite value that a query sees gives that infinity, NaN or both infinities give NaN."""
import pytest
import torch

import serving_ref as ref
import varlen_gated_delta_gb300 as gdn
from test_gpu_attention import BF16, DEV, F32, _lib, check, i32, make_paged, run_varlen  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def same_kind(got, want, what=""):
    """The same values are +inf, -inf and NaN."""
    got = got.detach().cpu().double()
    for name, kind in (("+inf", lambda x: x == INF), ("-inf", lambda x: x == -INF), ("NaN", torch.isnan)):
        bad = kind(got) != kind(want)
        assert not bool(bad.any()), f"{what}: {int(bad.sum())} values differ in being {name}"


def put(v, where):
    """Values into v[key, head, channel], by where(key)."""
    for key, head, channel, x in ((2, 0, 1, INF), (2, 0, 3, -INF), (40, 0, 3, INF), (63, 1, 2, -INF), (64, 1, 5, NAN),
                                  (100, 0, 9, -INF), (130, 1, 0, INF), (200, 0, 6, -INF), (290, 1, 7, INF)):
        at = where(key)
        if at is not None:
            v[at + (head, channel)] = x


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [16, 64, 100, 128, 256])
def test_varlen_kinds(dt, D):
    def edit(q, k, v):
        put(v, lambda key: (key + 20,))          # (the second sequence)
    lens = [20, 300, 31]
    q, k, v, out = run_varlen(lens, 4, 2, D, dt, seed=D, edit=edit)
    want, _ = ref.attention(q[20:320], k[20:320], v[20:320])
    same_kind(out[20:320], want)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [16, 64, 128, 256])
@pytest.mark.parametrize("news,kvs,pages", [([1, 1], [300, 41], 20), ([1, 1], [300, 41], 200), ([6, 3], [300, 131], 20),
                                            ([90, 20], [300, 131], 20), ([90, 20], [300, 131], 200)], ids=str)
def test_paged_kinds(dt, D, news, kvs, pages):
    q, kc, vc, table = make_paged(news, kvs, 4, 2, D, 16, dt, max_pages=pages)
    for b in range(2):
        put(vc, lambda key: (int(table[b, key // 16]), key % 16) if key < kvs[b] else None)
    out = torch.empty_like(q)
    gdn.gdn_attention_paged(q, kc, vc, i32(table), i32(kvs), i32([0, news[0], sum(news)]), max_q=max(news), out=out)
    at = 0
    for b, (n, kv) in enumerate(zip(news, kvs)):
        want, mag = ref.attention(q[at:at + n], ref.cached_rows(kc, table[b], kv), ref.cached_rows(vc, table[b], kv))
        check(out[at:at + n], want, mag, dt, str(b))
        same_kind(out[at:at + n], want, str(b))
        at += n
    gdn.gdn_attention_status()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_fp32_values_at_the_end_of_the_range_stay_finite(D):
    """One value of each such channel, so that no sum passes the range."""
    def edit(q, k, v):
        for key, c, x in ((5, 0, 3.4028e38), (70, 1, -3.4028e38), (199, 2, 3.4028234e38)):
            v[:, :, c] = 0
            v[key, :, c] = x
    q, k, v, out = run_varlen([200], 4, 2, D, F32, seed=D, edit=edit)
    assert bool(torch.isfinite(out).all())
