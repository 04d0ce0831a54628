"""gdn_qk_norm_rope against a plain 64-bit form.

Tolerances: fp32 arithmetic on values rounded once at the end.  A value is a few
products and one sum of two (relative error some 2^-21 of the head's largest value
with the mean of squares and the reciprocal root), so fp32 outputs are held to
4e-6 of the head's largest value and bf16 outputs to that plus half a bf16 step (2^-8
relative, the rounding's own bound being 2^-9)."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import varlen_gated_delta_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
SENTINEL = 777.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from varlen_gated_delta_gb300 import build
    build.build()
    gdn.load_library()


def _table(P, R):
    a = np.arange(P)[:, None] * 10000.0 ** (-np.arange(R // 2) * 2.0 / max(R, 1))[None, :]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).to(DEV)


def _close(got, want, dt, head_max):
    err = (got.detach().cpu().double() - want).abs()
    tol = 4e-6 * head_max + (2.0 ** -8 * want.abs() if dt == BF16 else 0.0)
    assert bool((err <= tol).all()), f"max error {float(err.max()):.3e}"


def _inputs(N, H, HKV, D, R, dt, seed, row_pad=0, P=50):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    W = (H + 2 * HKV) * D
    qkv = r(N, W + row_pad).to(dt)[:, :W]
    pos = torch.randint(0, P, (N,), generator=g, device=DEV, dtype=torch.int32)
    return qkv, (_table(P, R) if R else None), (pos if R else None), 1 + 0.3 * r(D), 1 + 0.3 * r(D)


def _want(qkv, table, pos, qw, kw, H, HKV, D, style, eps):
    x = qkv.reshape(qkv.shape[0], H + 2 * HKV, D)
    row = None if table is None else table[pos.long()]
    return (ref.norm_rope(x[:, :H], qw, eps, row, style), ref.norm_rope(x[:, H:H + HKV], kw, eps, row, style),
            x[:, H + HKV:])


SHAPES = [  # N, H, HKV, D, R, row padding
    (1, 4, 1, 128, 128, 0), (7, 32, 8, 128, 128, 0), (33, 16, 16, 64, 32, 0), (5, 8, 2, 256, 64, 0),
    (257, 3, 1, 128, 2, 0),                 # two rotated channels: no whole vector
    (9, 4, 2, 128, 96, 0),                  # not a power of two
    (6, 6, 2, 80, 40, 0), (4, 2, 1, 37, 12, 0), (3, 4, 4, 16, 0, 0),
    (11, 5, 5, 64, 64, 24),                 # rows further apart
    (11, 4, 2, 64, 64, 1),                  # and misaligned
    (2, 1, 1, 1, 0, 0), (2, 2, 1, 2, 2, 0), (700, 8, 2, 128, 64, 0),
]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("style", [gdn.GDN_ROPE_HALF, gdn.GDN_ROPE_PAIRS])
@pytest.mark.parametrize("N,H,HKV,D,R,pad", SHAPES)
def test_norm_and_rotation_match(dt, style, N, H, HKV, D, R, pad):
    qkv, table, pos, qw, kw = _inputs(N, H, HKV, D, R, dt, N + D, pad)
    q, k = gdn.gdn_qk_norm_rope(qkv, table, pos, H=H, HKV=HKV, D=D, q_weight=qw, k_weight=kw, eps=1e-5, style=style)
    wq, wk, _ = _want(qkv, table, pos, qw, kw, H, HKV, D, style, 1e-5)
    _close(q, wq, dt, wq.abs().amax(-1, keepdim=True))
    _close(k, wk, dt, wk.abs().amax(-1, keepdim=True))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256, 100])
def test_without_weights_only_the_rotation_is_applied(dt, D):
    qkv, table, pos, _, _ = _inputs(5, 4, 2, D, 32, dt, 3)
    q, k = gdn.gdn_qk_norm_rope(qkv, table, pos, H=4, HKV=2, D=D)
    wq, wk, _ = _want(qkv, table, pos, None, None, 4, 2, D, 0, 0.0)
    _close(q, wq, dt, wq.abs().amax(-1, keepdim=True))
    _close(k, wk, dt, wk.abs().amax(-1, keepdim=True))
    assert torch.equal(q[..., 32:], qkv.view(5, 8, D)[:, :4, 32:])     # unrotated channels bit for bit


def test_a_zero_head_stays_zero():
    qkv = torch.zeros(3, 4 * 128, device=DEV, dtype=BF16)
    one = torch.ones(128, device=DEV)
    q, k = gdn.gdn_qk_norm_rope(qkv, H=2, HKV=1, D=128, q_weight=one, k_weight=one, eps=1e-6)
    assert not q.any() and not k.any()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D,R", [(128, 128), (64, 32), (96, 96), (50, 10)])
@pytest.mark.parametrize("packed_k", [False, True])
def test_cache_slots(dt, D, R, packed_k):
    """k and v land in their slots; slots out of range write nothing; others keep their rows."""
    N, H, HKV, pages, ps = 37, 4, 2, 5, 9
    qkv, table, pos, qw, kw = _inputs(N, H, HKV, D, R, dt, 8)
    slots = torch.from_numpy(np.random.RandomState(5).permutation(pages * ps)[:N].astype(np.int32)).to(DEV)
    slots[3], slots[10], slots[11] = -1, pages * ps, 2**31 - 1
    kc = torch.full((pages, ps, HKV, D), SENTINEL, device=DEV, dtype=dt)
    vc = torch.full((pages, ps, HKV, D), SENTINEL, device=DEV, dtype=dt)
    k = torch.empty((N, HKV, D), device=DEV, dtype=dt) if packed_k else None
    q, k2 = gdn.gdn_qk_norm_rope(qkv, table, pos, H=H, HKV=HKV, D=D, q_weight=qw, k_weight=kw, k=k, slots=slots,
                                 k_cache=kc, v_cache=vc)
    wq, wk, wv = _want(qkv, table, pos, qw, kw, H, HKV, D, 0, 1e-6)
    _close(q, wq, dt, wq.abs().amax(-1, keepdim=True))
    assert (k2 is None) == (not packed_k)
    if packed_k:
        _close(k, wk, dt, wk.abs().amax(-1, keepdim=True))
    left = torch.ones(pages * ps, dtype=torch.bool)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * ps:
            left[s] = False
            _close(kc.view(-1, HKV, D)[s], wk[t], dt, wk[t].abs().amax(-1, keepdim=True))
            assert torch.equal(vc.view(-1, HKV, D)[s], wv[t])
    for c in (kc, vc):
        assert bool((c.view(-1, HKV, D).cpu()[left] == SENTINEL).all())


@pytest.mark.parametrize("D", [128, 50])
def test_a_token_outside_the_position_table_is_skipped(D):
    qkv, table, pos, qw, kw = _inputs(6, 4, 2, D, 10, BF16, 9)
    pos[1], pos[4] = -1, 50
    q = torch.full((6, 4, D), SENTINEL, device=DEV, dtype=BF16)
    k = torch.full((6, 2, D), SENTINEL, device=DEV, dtype=BF16)
    gdn.gdn_qk_norm_rope(qkv, table, pos, H=4, HKV=2, D=D, q_weight=qw, k_weight=kw, q=q, k=k,
                         style=gdn.GDN_ROPE_PAIRS)
    for t in range(6):
        kept = bool((q[t] == SENTINEL).all()) and bool((k[t] == SENTINEL).all())
        assert kept == (t in (1, 4))


def test_cache_elements_past_32_bits():
    """A slot whose element offset exceeds 2^32 (a cache of 4.3e9 bf16 values)."""
    H, HKV, D, ps = 16, 16, 256, 64
    pages = (1 << 32) // (ps * HKV * D) + 2
    kc = torch.zeros((pages, ps, HKV, D), device=DEV, dtype=BF16)
    vc = torch.zeros((pages, ps, HKV, D), device=DEV, dtype=BF16)
    qkv, table, pos, qw, kw = _inputs(2, H, HKV, D, 64, BF16, 4)
    slots = torch.tensor([pages * ps - 1, 5], dtype=torch.int32, device=DEV)
    gdn.gdn_qk_norm_rope(qkv, table, pos, H=H, HKV=HKV, D=D, q_weight=qw, k_weight=kw, slots=slots, k_cache=kc,
                         v_cache=vc)
    _, wk, wv = _want(qkv, table, pos, qw, kw, H, HKV, D, 0, 1e-6)
    for t, s in enumerate(slots.tolist()):
        _close(kc.view(-1, HKV, D)[s], wk[t], BF16, wk[t].abs().amax(-1, keepdim=True))
        assert torch.equal(vc.view(-1, HKV, D)[s], wv[t])
    assert int(torch.count_nonzero(vc.view(-1, HKV * D).any(-1))) == 2
