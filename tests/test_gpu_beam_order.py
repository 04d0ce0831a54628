"""The order of beams whose totals are equal, or nearly."""
import pytest
import torch

import varlen_gated_delta_gb300 as gdn

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("V,std", [(9001, 1.0), (32768, 1.0), (131072, 2.0)])
def test_totals_that_nearly_agree(V, std):
    """Pairs of beams whose best totals are 2^-24 to 2^-22 apart come in the order of their totals in 64 bits."""
    # A term's exponent is rounded to 2^-22 at most (in nats, for terms down to e^-11 of the largest) and its exponential to
    # 2^-22; such errors of V terms of about one size average out to some 2^-22 / sqrt(V / 3) <= 2^-27 here.  What all terms
    # share, the rounding of log2(e) to 2^-26, moves a row's log sum by that times the distance of its largest logit from the
    # bulk of the sum: two rows' distances differ by less than 3.  So 2^-24 is more than the difference of two rows' errors.
    gen = torch.Generator(device="cuda").manual_seed(V)
    G = 256 if V < 100000 else 64
    x = torch.randn(2 * G, V, generator=gen, device="cuda") * std
    best = (x.double().amax(1) - torch.logsumexp(x.double(), 1)).view(G, 2)
    apart = 2.0 ** -24 * (1 + 3 * torch.rand(G, generator=gen, device="cuda", dtype=torch.float64))
    sign = torch.where(torch.rand(G, generator=gen, device="cuda") < 0.5, 1.0, -1.0).double()
    # totals near -1/2: scores of about a unit, whose own rounding is taken into account
    scores = torch.stack([-0.5 - best[:, 0], -0.5 - best[:, 1] + sign * apart], 1).float()
    total = scores.double() + best
    some = (total[:, 0] - total[:, 1]).abs() >= 2.0 ** -24
    assert int(some.sum()) > G // 4
    _, parents, _, _ = gdn.gdn_beam_select(x, scores, n=2)
    second = total[:, 1] > total[:, 0]
    first = parents[:, 0] - 2 * torch.arange(G, device="cuda", dtype=I32)
    assert torch.equal(first[some], second[some].int())


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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dead", [-1e4, -1e9, -3.4e38, torch.finfo(F32).min])
@pytest.mark.parametrize("V", [40, 3001, 140001])
def test_dead_beams_with_finite_scores(V, dead, dtype):
    """The first step of a search whose dead beams have a large negative score instead of -inf."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    K, n = 8, 16
    logits = (torch.randn(2 * K, V, generator=gen, device="cuda") * 3).to(dtype)
    scores = torch.full((2, K), dead, device="cuda")
    scores[0, 0] = scores[1, 3] = 0.0
    logits[K + 3, 5:] = -float("inf")  # the live beam of the second group has five continuations
    tokens, parents, totals, _ = gdn.gdn_beam_select(logits, scores, n=n)
    # the definition: by total, then the lowest beam; within a beam by logit, then the lowest token
    for g in range(2):
        found = []
        for k in range(K):
            row = logits[g * K + k].double()
            total = float(scores[g, k]) + (row - torch.logsumexp(row, 0))
            best = torch.sort(row, descending=True, stable=True).indices[:n].tolist()
            found += [(-float(total[t]), k, i, t) for i, t in enumerate(best) if row[t] > -float("inf")]
        found = sorted(found)[:n]
        assert parents[g].tolist() == [g * K + f[1] for f in found]
        assert tokens[g].tolist() == [f[3] for f in found]
        want = torch.tensor([-f[0] for f in found], dtype=torch.float64)
        # one rounding to fp32, and a sum of fp32 exponentials that is 2^-20 off at most
        assert bool(((totals[g].cpu().double() - want).abs() <= want.abs() * 2.0 ** -24 + 2.0 ** -20).all())
