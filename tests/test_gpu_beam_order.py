"""The order of beams whose totals are equal, or nearly."""
import pytest
import torch

import varlen_gated_delta_gb300 as gdn

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1001, 4099, 32771, 50001, 131073])
def test_equal_rows_stay_in_order(V, dtype):
    """Beams with the same logits and scores have the same totals, wherever in memory their rows begin."""
    G, K = (48 if V < 50000 else 16), 8
    gen = torch.Generator(device="cuda").manual_seed(V)
    rows = torch.randn(G, V, generator=gen, device="cuda").to(dtype)
    logits = rows.repeat_interleave(K, 0)
    scores = (-torch.rand(G, 1, generator=gen, device="cuda")).expand(G, K).contiguous()
    tokens, parents, totals, _ = gdn.gdn_beam_select(logits, scores)
    best, at = torch.sort(rows.float(), dim=1, descending=True, stable=True)
    for g in range(G):  # by logit, then beam, then token
        found = sorted((-x, k, t) for x, t in zip(best[g, :K].tolist(), at[g, :K].tolist()) for k in range(K))[:K]
        assert parents[g].tolist() == [g * K + f[1] for f in found]
        assert tokens[g].tolist() == [f[2] for f in found]
        same = [f[0] == found[0][0] for f in found]
        assert len({x for x, s in zip(totals[g].tolist(), same) if s}) == 1
