"""Selection of beams and the reordering of states on the GPU."""
import pytest
import torch

import beam_ref
import varlen_gated_delta_gb300 as gdn

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _check(logits, scores, n, got, finished=None, end=-1, keep=False):
    want = beam_ref.beam_select(logits, scores, n, finished, end, keep)
    tokens, parents, totals, done = got
    assert tokens.tolist() == [[f[2] for f in g] for g in want]
    assert parents.tolist() == [[f[1] for f in g] for g in want]
    want_totals = torch.tensor([[f[0] for f in g] for g in want], dtype=torch.float64)
    # one rounding to fp32 (2^-24), and a sum of fp32 exponentials that is 2^-20 off at most
    tol = want_totals.abs().nan_to_num(posinf=0, neginf=0) * 2.0 ** -24 + 2.0 ** -20
    same = totals.cpu().double() == want_totals
    assert bool((same | ((totals.cpu().double() - want_totals).abs() <= tol)).all())
    if done is not None:
        assert done.bool().tolist() == [[f[3] for f in g] for g in want]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("G,K,V,n", [
    (1, 1, 1, 1), (1, 4, 7, 4), (2, 3, 100, 5), (3, 4, 2048, 4), (1, 4, 32768, 8), (2, 8, 50001, 8), (5, 16, 4099, 32), (1, 2, 131072, 100),
    (40, 5, 30007, 5), (1, 128, 300, 128), (1, 1, 200000, 1)])
def test_select(G, K, V, n, dtype):
    gen = torch.Generator(device="cuda").manual_seed(V + n)
    # (fp32 values: no two are as near as the sums' errors; bf16: many are equal, and ties go by place)
    logits = (torch.randn(G * K, V, generator=gen, device="cuda") * 3).to(dtype)
    scores = -4 * torch.rand(G, K, generator=gen, device="cuda")
    _check(logits, scores, n, gdn.gdn_beam_select(logits, scores, n=n))
    if n == K:
        finished = torch.rand(G, K, generator=gen, device="cuda") < 0.4
        end = V // 2
        for keep in (False, True):
            _check(logits, scores, n, gdn.gdn_beam_select(logits, scores, finished=finished, end_token=end, keep_rows=keep), finished,
                   end, keep)
        _check(logits, scores, n, gdn.gdn_beam_select(logits, scores, keep_rows=True), keep=True)


def test_equal_logits_and_equal_beams():
    """Ties go to the lowest beam and token, however many there are."""
    for V in (33, 4096, 40000):
        logits = torch.zeros(8, V, device="cuda", dtype=BF16)
        scores = torch.zeros(2, 4, device="cuda")
        _check(logits, scores, 6, gdn.gdn_beam_select(logits, scores, n=6))
        logits[:, V // 3:] = 2.0
        _check(logits, scores, 6, gdn.gdn_beam_select(logits, scores, n=6))
        logits[:, ::2] *= -0.0  # negative zeros are zeros
        _check(logits, scores, 6, gdn.gdn_beam_select(logits, scores, n=6))


@pytest.mark.parametrize("V", [50, 9000])
def test_masked_logits_and_beams(V):
    inf = float("inf")
    gen = torch.Generator(device="cuda").manual_seed(V)
    logits = torch.randn(8, V, generator=gen, device="cuda")
    logits[0] = -inf                       # nothing may follow
    logits[1, 3:] = -inf                   # three may
    logits[2, 5] = float("nan")            # no candidate
    logits[3, 6] = inf                     # a row without probabilities
    logits[4:, 2:] = -inf                  # a group with eight in all
    scores = torch.tensor([[0.0, -1.0, -inf, -0.5], [-1.0, -inf, float("nan"), -2.0]], device="cuda")
    for n in (4, 6):
        _check(logits, scores, n, gdn.gdn_beam_select(logits, scores, n=n))
    # masks of the type's lowest value, a whole row of them among others, and logits of any size
    for dtype in (F32, BF16):
        low = torch.finfo(dtype).min
        big = torch.randn(8, V, generator=gen, device="cuda").to(dtype)
        big[0], big[1, 4:], big[2, ::2], big[3] = low, low, low, big[3] * 1e6
        big[4], big[5, 7], big[6] = big[4] * 1e30, -low, big[6] + 3e4
        zero = torch.zeros(2, 4, device="cuda")
        _check(big, zero, 4, gdn.gdn_beam_select(big, zero))
    # the first step of a search: one live beam
    scores = torch.tensor([[0.0, -inf, -inf, -inf]], device="cuda")
    _check(logits[1:5], scores, 4, gdn.gdn_beam_select(logits[1:5], scores))
    # all at their end
    done = torch.ones(2, 4, dtype=torch.uint8, device="cuda")
    scores = torch.tensor([[-3.0, -1.0, -2.0, -1.0], [-1.0, -inf, -4.0, -0.5]], device="cuda")
    for keep in (False, True):
        _check(logits, scores, 4, gdn.gdn_beam_select(logits, scores, finished=done, end_token=7, keep_rows=keep), done, 7, keep)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [4, 160])
def test_long_rows_of_every_kind(rows, dtype):
    """Rows that a CTA goes through in several pieces: rising, falling, equal, masked at the front, largest at the end."""
    V, K = 150001, 4
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, V, generator=gen, device="cuda")
    ramp = torch.arange(V, device="cuda") / 1000
    x[0], x[1], x[2, :] = ramp, ramp.flip(0), 2.0
    x[3, :100000] = -float("inf")
    x[3, 100003:] = -float("inf")
    if rows > 4:
        x[4, -3:] += 60                                   # the reference moves in the last piece
        x[5, 20000:] += 30
        x[6, ::2] = -float("inf")
        x[7, 140000] = float("nan")
        x[8] = torch.where(ramp > 100, 3.0, -float("inf"))
        x[9, 70000:] = 0.0
        x[10, 16384 * 3 - 2:16384 * 3 + 2] = 9.0          # equal ones across a border
    x = x.to(dtype)
    scores = -torch.rand(rows // K, K, generator=gen, device="cuda")
    for n in (4, 40, 128):
        _check(x, scores, n, gdn.gdn_beam_select(x, scores, n=n))


def test_rows_of_any_stride_and_outputs_in_place():
    gen = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn(12, 5003, generator=gen, device="cuda").to(BF16)
    for first in range(8):
        logits = wide[:, first:first + 4990]
        scores = -torch.rand(3, 4, generator=gen, device="cuda")
        _check(logits, scores, 4, gdn.gdn_beam_select(logits, scores))
    done = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    done[1, 2] = True
    was, was_done = scores.clone(), done.clone()
    ws = torch.full((gdn.gdn_beam_select_workspace_bytes(3, 4, 4990, 4),), 255, dtype=torch.uint8, device="cuda")
    got = gdn.gdn_beam_select(logits, scores, finished=done, end_token=9, scores_out=scores, finished_out=done, workspace=ws)
    assert got[2] is scores and got[3] is done and done.dtype == torch.bool
    _check(logits, was, 4, got, was_done, 9)


def test_select_refusals():
    logits, scores = torch.zeros(8, 40, device="cuda"), torch.zeros(2, 4, device="cuda")
    flags = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    for bad in (dict(logits=logits[:7]), dict(logits=logits.half()), dict(logits=logits.T), dict(scores=scores.double()), dict(n=0),
                dict(n=129), dict(n=3, keep_rows=True), dict(finished=flags), dict(finished=flags, end_token=40), dict(finished=flags[:1]),
                dict(finished=flags.int(), end_token=1), dict(scores_out=scores, n=3), dict(logits=logits[:, :0]),
                dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), dict(tokens=flags), dict(scores=scores.cpu())):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_beam_select(**dict(dict(logits=logits, scores=scores), **bad))


# ---------------------------------------------------------------- states

@pytest.mark.parametrize("B", [1, 2, 7, 64, 300, 4096])
def test_reorder(B):
    gen = torch.Generator(device="cuda").manual_seed(B)
    width = 1 if B > 1000 else 5
    states = [torch.randn(B, width, 33, 16, generator=gen, device="cuda"),                       # 16-byte accesses
              torch.randn(B, 77, 3, generator=gen, device="cuda").to(BF16),                      # 2
              torch.randint(0, 255, (B, 13), generator=gen, device="cuda", dtype=torch.uint8),   # 1
              torch.randn(B, 3, generator=gen, device="cuda"),                                   # 4
              torch.randn(B, 0, 4, generator=gen, device="cuda"),
              torch.randint(0, 99, (B, 1001), generator=gen, device="cuda")]                     # 8
    for kind in ("any", "turn", "one", "same", "outside"):
        parents = {"any": torch.randint(0, B, (B,), generator=gen, device="cuda"), "turn": (torch.arange(B, device="cuda") + 1) % B,
                   "one": torch.zeros(B, device="cuda"), "same": torch.arange(B, device="cuda"),
                   "outside": torch.randint(-2, B + 2, (B,), generator=gen, device="cuda")}[kind].to(I32)
        p = parents.long()
        p = torch.where((p < 0) | (p >= B), torch.arange(B, device="cuda"), p)
        want = [t[p] for t in states]
        gdn.gdn_state_reorder(states, parents)
        for t, w in zip(states, want):
            assert torch.equal(t, w), kind


def test_reorder_of_odd_addresses_and_many_tensors():
    room = torch.arange(4 * 1001 + 3, dtype=torch.uint8, device="cuda")
    view = room[3:].view(4, 1001)
    before, want = room.clone(), view[[2, 2, 0, 1]].clone()
    gdn.gdn_state_reorder([view], torch.tensor([2, 2, 0, 1], dtype=I32, device="cuda"))
    assert torch.equal(view, want) and torch.equal(room[:3], before[:3])
    many = [torch.randn(3, 65 + i, device="cuda") for i in range(64)]
    want = [t[[1, 1, 0]] for t in many]
    parents = torch.tensor([1, 1, 0], dtype=I32, device="cuda")
    gdn.gdn_state_reorder(many, parents)
    assert all(torch.equal(t, w) for t, w in zip(many, want))
    gdn.gdn_state_reorder([], parents)
    big = torch.randn(8, 1 << 20, device="cuda")
    want = big[[7, 0, 0, 3, 2, 2, 6, 1]]
    gdn.gdn_state_reorder((big,), torch.tensor([7, 0, 0, 3, 2, 2, 6, 1], dtype=I32, device="cuda"))
    assert torch.equal(big, want)


def test_reorder_refusals():
    a, parents = torch.zeros(4, 6, device="cuda"), torch.zeros(4, dtype=I32, device="cuda")
    for states, p in (([a, a], parents), ([a[:, :3]], parents), ([a, torch.zeros(3, 6, device="cuda")], parents), ([a], parents[:3]),
                      ([a], parents.long()), ([a] * 65, parents), ([torch.zeros(4097, 1, device="cuda")], parents),
                      ([torch.zeros((), device="cuda")], parents), ([a.cpu()], parents), ([a], parents.cpu())):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_state_reorder(states, p)
    with pytest.raises(TypeError):
        gdn.gdn_state_reorder(a.sum, parents)
    with pytest.raises(TypeError):
        gdn.gdn_state_reorder([a, 3], parents)
