"""Non-finite values among long prompts and histories: they reach the queries that see them, and nothing else of
the call changes.  Compared bit for bit with the call that has zeros in their places."""
import numpy as np
import pytest
import torch

import varlen_gated_delta_gb300 as gdn
from test_gpu_attention import BF16, DEV, _lib, i32, make_paged  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def same(got, want):
    """Bit for bit, NaN for NaN."""
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_slices_over_a_long_history_with_non_finite_values(D):
    """They reach the queries that see them and change nothing else, whatever the history's length: against the call
    with zeros in their places, every other value of every request is the same."""
    news, kvs, ps = [200, 130], [65536, 500], 64
    q, kc, vc, table = make_paged(news, kvs, 4, 2, D, ps, BF16)
    places = ((kvs[0] - 40, 0, 3, NAN), (kvs[0] - 150, 1, 5, INF))
    args = (i32(table), i32(kvs), i32([0, 200, 330]))
    for t, head, c, _ in places:
        vc[int(table[0, t // ps]), t % ps, head, c] = 0
    want = gdn.gdn_attention_paged(q, kc, vc, *args, max_q=200)
    assert bool(torch.isfinite(want).all())
    for t, head, c, x in places:
        vc[int(table[0, t // ps]), t % ps, head, c] = x
        want[t - kvs[0] + 200:200, 2 * head:2 * head + 2, c] = x
    same(gdn.gdn_attention_paged(q, kc, vc, *args, max_q=200), want)
    gdn.gdn_attention_status()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,HKV", [(8, 2), (3, 3)])
def test_long_prompts_with_non_finite_values(D, H, HKV):
    """As above, with several items of work for each CTA: a prompt of 20000 tokens between others."""
    lens, G = [50, 20000, 3000, 77], H // HKV
    offs = np.concatenate([[0], np.cumsum(lens)])
    g = torch.Generator(device=DEV)
    g.manual_seed(D)
    q, k, v = (torch.randn(int(offs[-1]), h, D, generator=g, device=DEV).to(BF16) for h in (H, HKV, HKV))
    places = ((1, 19990, 1, 2, NAN), (1, 64, 0, 3, INF), (2, 1, 1, 0, -INF), (2, 2999, 0, 7, NAN), (3, 30, 0, 1, INF))
    for b, t, head, c, _ in places:
        v[offs[b] + t, head, c] = 0
    want = gdn.gdn_attention_varlen(q, k, v, i32(offs))
    assert bool(torch.isfinite(want).all())
    for b, t, head, c, x in places:
        v[offs[b] + t, head, c] = x
        want[offs[b] + t:offs[b + 1], head * G:(head + 1) * G, c] = x
    same(gdn.gdn_attention_varlen(q, k, v, i32(offs)), want)
    gdn.gdn_attention_status()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_prompt_whose_values_are_all_nan_beside_others(D):
    lens = [600, 1500, 300]
    g = torch.Generator(device=DEV)
    g.manual_seed(D)
    q, k, v = (torch.randn(2400, h, D, generator=g, device=DEV).to(BF16) for h in (4, 2, 2))
    want = gdn.gdn_attention_varlen(q, k, v, i32([0, 600, 2100, 2400]))
    v[600:2100] = NAN
    want[600:2100] = NAN
    same(gdn.gdn_attention_varlen(q, k, v, i32([0, 600, 2100, 2400])), want)
    gdn.gdn_attention_status()
