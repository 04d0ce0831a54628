"""gdn_attention_varlen and gdn_attention_paged against a plain 64-bit softmax.

Tolerances, per output value, with M = sum_j p_j |v_j| from the 64-bit form:
- bf16: probabilities rounded to bf16 (relative 2^-9 each, so 2^-9 M in the sum) and the
  output rounded to bf16 (2^-9 |o|); doubled: 2^-8 (M + |o|).
- fp32: a score is a sum of D products in fp32, off by at most about D 2^-24 scale |q| |k|
  (1e-5 .. 1e-4 for the spreads here), which enters p relatively: 1e-4 M; the errors are
  random, so the relative 2-norm is held to 1e-5."""
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


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64), dtype=torch.int32, device=DEV)


def rand(g, *shape, dt=BF16, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dt)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def check(got, want, mag, dt, what=""):
    got = got.detach().cpu().double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: finite places differ"
    ok = torch.isfinite(want)
    err = torch.where(ok, (got - want).abs(), torch.zeros_like(want))
    tol = 2.0 ** -8 * (mag + want.abs()) if dt == BF16 else 1e-4 * mag
    assert bool((err <= torch.where(ok, tol + 1e-30, torch.full_like(tol, 1.0))).all()), \
        f"{what}: max error {float(err.max()):.3e}"
    if dt == F32 and bool(ok.all()) and float(want.norm()) > 0:
        assert float((got - want).norm() / want.norm()) <= 1e-5, what


# ---------------------------------------------------------------- packed prompts

def run_varlen(lens, H, HKV, D, dt, seed=0, pad=(0, 0, 0), extra_rows=0, scale=0.0, edit=None, std=2.0):
    g = gen(seed)
    offs = np.concatenate([[0], np.cumsum(lens)])
    N = int(offs[-1]) + extra_rows
    q = rand(g, N, H * D + pad[0], dt=dt, std=std)[:, :H * D].view(N, H, D) if pad[0] == 0 else \
        torch.as_strided(rand(g, N, H * D + pad[0], dt=dt, std=std), (N, H, D), (H * D + pad[0], D, 1))
    k, v = (torch.as_strided(rand(g, N, HKV * D + p, dt=dt), (N, HKV, D), (HKV * D + p, D, 1)) for p in pad[1:])
    if edit is not None:
        edit(q, k, v)
    out = torch.full((N, H, D), SENTINEL, device=DEV, dtype=dt)
    gdn.gdn_attention_varlen(q, k, v, i32(offs), scale=scale, out=out)
    for b in range(len(lens)):
        s, e = int(offs[b]), int(offs[b + 1])
        if e == s:
            continue
        want, mag = ref.attention(q[s:e], k[s:e], v[s:e], scale or None)
        check(out[s:e], want, mag, dt, f"sequence {b} of {lens}")
    assert bool((out[int(offs[-1]):] == SENTINEL).all())
    return q, k, v, out


LENS = [[1], [2, 1, 1], [0, 5, 0, 0, 64], [63, 65], [127, 128, 129], [255, 1, 256], [257, 300], [400, 3, 0, 513]]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_varlen_lengths(dt, lens):
    run_varlen(lens, 4, 2, 128, dt, seed=sum(lens))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("H,HKV,D", [(1, 1, 128), (8, 1, 64), (6, 2, 64), (4, 4, 256), (8, 2, 256), (5, 5, 96), (4, 2, 80),
                                     (2, 1, 16), (3, 1, 100), (2, 2, 37), (2, 1, 1), (4, 1, 192), (2, 1, 250)])
def test_varlen_heads(dt, H, HKV, D):
    run_varlen([130, 1, 270], H, HKV, D, dt, seed=D)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("pad", [(64, 0, 0), (0, 128, 256), (8, 8, 8), (1, 3, 5), (0, 0, 2)])
def test_varlen_token_strides(dt, pad):
    """Rows further apart than their width, also by amounts that break 16-byte alignment."""
    run_varlen([100, 40, 161], 4, 2, 64, dt, seed=7, pad=pad)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_varlen_rows_past_the_last_sequence_are_not_written(dt):
    run_varlen([70, 33], 4, 2, 128, dt, extra_rows=50)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("scale", [0.01, 1.0, -0.3])
def test_varlen_scale(dt, scale):
    """An explicit scale; 1.0 gives scores of spread 20, near one-hot rows."""
    run_varlen([90, 200], 2, 1, 128, dt, seed=5, scale=scale, std=1.0 if scale != 1.0 else 0.5)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_varlen_growing_scores(dt):
    """Keys whose scores grow along the sequence, so that the running maximum moves in every tile."""
    def edit(q, k, v):
        n = k.shape[0]
        q.copy_(torch.ones_like(q))
        k.copy_((torch.linspace(0, 8, n, device=DEV)[:, None, None] * torch.ones_like(k)).to(k.dtype))
    run_varlen([700], 2, 1, 64, dt, edit=edit)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256, 100])
def test_varlen_non_finite_values_reach_only_the_queries_that_see_them(dt, D):
    """inf and NaN in v: causal masks and sequence ends keep them from earlier queries and other sequences."""
    def edit(q, k, v):
        v[37, 0, 3] = float("inf")
        v[61, 0, 5] = float("nan")
        v[61, 1, :] = float("-inf")
        v[200, 1, 9] = float("nan")      # second sequence, second tile
        v[331, 0, 0] = float("inf")      # first token of the third sequence
    lens = [100, 230, 40]
    q, k, v, out = run_varlen(lens, 4, 2, D, dt, seed=11, edit=edit)
    assert bool(torch.isfinite(out[:37]).all()) and bool(torch.isfinite(out[101:200]).all())
    assert not bool(torch.isfinite(out[37:100, 0, 3]).any())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_varlen_non_finite_keys_reach_only_the_queries_that_see_them(dt, D):
    def edit(q, k, v):
        k[90, 0, 0] = float("nan")
        k[150, 1, 0] = float("inf")
    q, k, v, out = run_varlen([91, 120], 4, 2, D, dt, seed=12, edit=edit)
    assert bool(torch.isfinite(out[:90]).all())
    assert bool(torch.isfinite(out[91:150]).all())


@pytest.mark.parametrize("dt", [F32, BF16])
def test_varlen_malformed_sequences_are_skipped(dt):
    g = gen(3)
    q, k, v = (rand(g, 100, 2, 64, dt=dt) for _ in range(3))
    out = torch.full((100, 2, 64), SENTINEL, device=DEV, dtype=dt)
    gdn.gdn_attention_varlen(q, k, v, i32([0, 40, 30, 100, 140]), out=out)   # decreasing, then past N
    want, mag = ref.attention(q[:30], k[:30], v[:30])
    check(out[:30], want, mag, dt)
    out.fill_(SENTINEL)
    gdn.gdn_attention_varlen(q, k, v, i32([0, 130]), out=out)
    assert bool((out == SENTINEL).all())


def test_varlen_many_short_sequences():
    lens = np.random.RandomState(2).randint(0, 4, 500).tolist()
    run_varlen(lens, 2, 1, 64, BF16)


@pytest.mark.parametrize("dt,D", [(F32, 128), (BF16, 128), (BF16, 64), (BF16, 256)])
def test_varlen_is_repeatable_and_independent_of_the_batch(dt, D):
    g = gen(9)
    lens = [300, 77, 512]
    N = sum(lens)
    q, k, v = rand(g, N, 8, D, dt=dt), rand(g, N, 2, D, dt=dt), rand(g, N, 2, D, dt=dt)
    a = gdn.gdn_attention_varlen(q, k, v, i32([0, 300, 377, 889]))
    assert torch.equal(a, gdn.gdn_attention_varlen(q, k, v, i32([0, 300, 377, 889])))
    one = gdn.gdn_attention_varlen(q[300:377], k[300:377], v[300:377], i32([0, 77]))
    assert torch.equal(a[300:377], one)


# ---------------------------------------------------------------- paged cache

def make_paged(news, kvs, H, HKV, D, ps, dt, seed=0, garbage=float("nan"), max_pages=None, std=2.0):
    """A cache whose unused slots hold `garbage`, with pages in random order."""
    g = gen(seed)
    rs = np.random.RandomState(seed)
    B = len(news)
    used = [-(-max(kv, 0) // ps) for kv in kvs]
    M = max_pages or max(max(used), 1)
    pages = sum(used) + 3
    order = rs.permutation(pages).tolist()
    table = np.full((B, M), -5)
    kc = torch.full((pages, ps, HKV, D), garbage, device=DEV, dtype=dt)
    vc = torch.full((pages, ps, HKV, D), garbage, device=DEV, dtype=dt)
    for b in range(B):
        for i in range(used[b]):
            table[b, i] = order.pop()
            n = min(ps, kvs[b] - i * ps)
            kc[table[b, i], :n] = rand(g, n, HKV, D, dt=dt)
            vc[table[b, i], :n] = rand(g, n, HKV, D, dt=dt)
    N = sum(news)
    q = rand(g, N, H, D, dt=dt, std=std)
    return q, kc, vc, table


def check_paged(out, q, kc, vc, table, news, kvs, dt, what="", scale=None):
    at = 0
    for b, (n, kv) in enumerate(zip(news, kvs)):
        if n:
            k, v = ref.cached_rows(kc, table[b], kv), ref.cached_rows(vc, table[b], kv)
            want, mag = ref.attention(q[at:at + n], k, v, scale)
            check(out[at:at + n], want, mag, dt, f"{what} sequence {b}: {n} of {kv}")
        at += n


def run_paged(news, kvs, H, HKV, D, ps, dt, seed=0, max_q=None, **kw):
    q, kc, vc, table = make_paged(news, kvs, H, HKV, D, ps, dt, seed, **kw)
    out = torch.full(q.shape, SENTINEL, device=DEV, dtype=dt)
    gdn.gdn_attention_paged(q, kc, vc, i32(table), i32(kvs), i32(np.concatenate([[0], np.cumsum(news)])),
                            max_q=max(news) if max_q is None else max_q, out=out)
    check_paged(out, q, kc, vc, table, news, kvs, dt)
    return out


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ps", [1, 7, 16, 64, 100, 256])
def test_paged_single_tokens(dt, ps):
    """Decode steps over histories that end inside, at and just past pages and tiles."""
    run_paged([1] * 12, [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300, 515], 8, 2, 128, ps, dt, seed=ps)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("H,HKV,D", [(1, 1, 128), (8, 1, 64), (16, 1, 128), (32, 2, 64), (64, 1, 128), (6, 2, 256), (5, 5, 96),
                                     (4, 2, 80), (3, 1, 100), (2, 2, 37), (48, 2, 128), (16, 2, 256), (100, 1, 64), (2, 1, 8)])
def test_paged_heads(dt, H, HKV, D):
    run_paged([1, 1, 1], [1, 77, 402], H, HKV, D, 16, dt, seed=D)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("news", [[2, 3, 5], [8, 1, 8], [1, 0, 8], [4, 4, 4]])
@pytest.mark.parametrize("H,HKV,D", [(8, 2, 128), (4, 4, 64), (16, 2, 256), (8, 1, 128)])
def test_paged_drafts(dt, news, H, HKV, D):
    """Up to 8 new tokens, as the delta layer's capture takes, on short and long histories."""
    run_paged(news, [n + h for n, h in zip(news, (0, 61, 350))], H, HKV, D, 16, dt, seed=sum(news))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ps", [16, 24, 64, 256])
@pytest.mark.parametrize("H,HKV,D", [(4, 2, 128), (2, 1, 64), (4, 1, 256), (2, 2, 96)])
def test_paged_prompt_slices(dt, ps, H, HKV, D):
    """Slices of prompts beside single tokens and drafts in one call."""
    news = [1, 130, 300, 0, 65, 3]
    run_paged(news, [200, 130, 437, 50, 66, 3], H, HKV, D, ps, dt, seed=ps + D)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_paged_long_history_few_sequences(dt, D):
    """Histories long enough to be split over many CTAs and joined."""
    run_paged([1, 1], [5003, 9], 8, 2, D, 64, dt, seed=1)
    run_paged([1], [9000], 4, 4, D, 64, dt, seed=2)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("H,HKV,D", [(8, 2, 128), (3, 1, 64), (4, 4, 64), (4, 1, 256), (2, 2, 96)])
@pytest.mark.parametrize("news,history", [([130], [3000]), ([70, 3, 200], [2900, 2500, 0]), ([65, 129], [127, 4000])])
def test_paged_slices_over_long_histories(dt, H, HKV, D, news, history):
    """Few items over many key tiles, which are then split; beside them sequences that see few keys or one tile."""
    run_paged(news, [n + h for n, h in zip(news, history)], H, HKV, D, 64, dt, seed=D + sum(news))


@pytest.mark.parametrize("H,HKV,D,news,history", [
    (8, 1, 128, [20, 9, 33], [0, 700, 63]), (16, 2, 256, [30, 12], [1500, 5]), (128, 1, 64, [2, 1, 3], [40, 0, 900]),
    (32, 1, 64, [5, 0, 3], [77, 10, 2000]), (4, 1, 96, [100, 17], [0, 333]), (4, 2, 128, [127, 33], [130, 1])])
def test_paged_short_slices_with_shared_heads(H, HKV, D, news, history):
    """Fewer tokens than a query tile has rows: the tile holds the heads of a group side by side."""
    run_paged(news, [n + h for n, h in zip(news, history)], H, HKV, D, 16, BF16, seed=H + D, max_pages=130)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_paged_split_slices_with_non_finite_values_and_rows_that_see_nothing(D):
    news, kvs = [100, 90], [2500, 20]
    q, kc, vc, table = make_paged(news, kvs, 4, 2, D, 16, BF16, max_pages=200)
    where = lambda b, t: (int(table[b, t // 16]), t % 16)
    vc[where(0, 2460)][0, 4] = float("nan")           # the 60th of the new tokens
    vc[where(0, 2499)][1, 5] = float("inf")
    kc[where(0, 2480)][1, 0] = float("nan")
    out = torch.full(q.shape, SENTINEL, device=DEV, dtype=BF16)
    gdn.gdn_attention_paged(q, kc, vc, i32(table), i32(kvs), i32([0, 100, 190]), max_q=100, out=out)
    check_paged(out, q, kc, vc, table, news, kvs, BF16)
    assert bool(torch.isfinite(out[:60]).all()) and not out[100:170].any()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("news", [[1, 1, 1, 1], [3, 8, 2, 1], [70, 3, 300, 1]])
def test_paged_rows_that_see_nothing_give_zero(dt, news):
    """Histories of no tokens, or of fewer than the new ones."""
    kvs = [0, 2, 1, 40]
    out = run_paged(news, kvs, 8, 2, 128, 16, dt)
    at = 0
    for n, kv in zip(news, kvs):
        assert not out[at:at + max(0, n - kv)].any()
        at += n


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n", [1, 5, 90])
def test_paged_malformed_sequences_are_skipped(dt, n):
    news, kvs = [n] * 4, [50 + n, 60 + n, 40 + n, 30 + n]
    q, kc, vc, table = make_paged(news, kvs, 4, 2, 64, 16, dt, max_pages=12)
    out = torch.full(q.shape, SENTINEL, device=DEV, dtype=dt)
    bad = list(kvs)
    bad[1], bad[2] = -1, 12 * 16 + 1                        # negative, and past the block table
    gdn.gdn_attention_paged(q, kc, vc, i32(table), i32(bad), i32(np.arange(5) * n), max_q=n, out=out)
    assert bool((out[n:3 * n] == SENTINEL).all())
    for b in (0, 3):
        check_paged(out[b * n:(b + 1) * n], q[b * n:(b + 1) * n], kc, vc, table[b:b + 1], [n], [kvs[b]], dt)
    out.fill_(SENTINEL)                                     # more new tokens than max_q says
    gdn.gdn_attention_paged(q, kc, vc, i32(table), i32(kvs), i32([0, n + 1, n + 1, 3 * n, 4 * n - 1]), max_q=n, out=out)
    assert bool((out[:n + 1] == SENTINEL).all())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n", [1, 90])
def test_paged_pages_outside_the_cache_read_as_zeros(dt, n):
    kvs = [70 + n, 300 + n]
    q, kc, vc, table = make_paged([n, n], kvs, 4, 2, 128, 16, dt)
    table[0, 1], table[1, 3], table[1, 7] = -1, kc.shape[0], 2**31 - 1
    out = torch.empty_like(q)
    gdn.gdn_attention_paged(q, kc, vc, i32(table), i32(kvs), i32([0, n, 2 * n]), max_q=n, out=out)
    check_paged(out, q, kc, vc, table, [n, n], kvs, dt)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_paged_non_finite_values_reach_only_the_queries_that_see_them(dt, D):
    for news, kvs in (([8, 5], [50, 133]), ([100, 7], [200, 133])):
        q, kc, vc, table = make_paged(news, kvs, 4, 2, D, 16, dt)
        where = lambda b, t: (int(table[b, t // 16]), t % 16)
        for b, t, x in ((0, kvs[0] - 3, float("nan")), (1, kvs[1] - 1, float("inf"))):
            vc[where(b, t)][0, 4] = x
        kc[where(0, kvs[0] - 1)][1, 0] = float("nan")
        out = torch.empty_like(q)
        gdn.gdn_attention_paged(q, kc, vc, i32(table), i32(kvs), i32([0, news[0], sum(news)]), max_q=max(news), out=out)
        check_paged(out, q, kc, vc, table, news, kvs, dt)
        assert bool(torch.isfinite(out[:news[0] - 3]).all()) and bool(torch.isfinite(out[news[0]:-1]).all())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [-0.2, 0.03])
@pytest.mark.parametrize("news", [[1, 1], [5, 2], [80, 3]])
def test_paged_scale_and_strided_queries(dt, D, scale, news):
    kvs = [n + h for n, h in zip(news, (130, 70))]
    q, kc, vc, table = make_paged(news, kvs, 8, 2, D, 16, dt)
    wide = torch.zeros(q.shape[0], 8 * D + 64, device=DEV, dtype=dt)
    wide[:, 64:] = q.view(q.shape[0], -1)
    view = wide[:, 64:].view(q.shape[0], 8, D) if q.shape[0] == 1 else \
        torch.as_strided(wide, q.shape, (8 * D + 64, D, 1), 64)
    out = gdn.gdn_attention_paged(view, kc, vc, i32(table), i32(kvs), i32([0, news[0], sum(news)]), max_q=max(news),
                                  scale=scale)
    check_paged(out, q, kc, vc, table, news, kvs, dt, scale=scale)
    gdn.gdn_attention_status()


def test_paged_padded_step():
    """A step of fixed size with fewer tokens: rows past offsets[B] and requests without tokens."""
    q, kc, vc, table = make_paged([1, 0, 1, 0, 2], [40, 33, 70, 0, 0], 8, 2, 128, 16, BF16)
    out = torch.full(q.shape, SENTINEL, device=DEV, dtype=BF16)
    gdn.gdn_attention_paged(q, kc, vc, i32(table), i32([40, 33, 70, 0, 0]), i32([0, 1, 1, 2, 2, 2]), max_q=1, out=out)
    check_paged(out[:2], q[:2], kc, vc, table[[0, 2]], [1, 1], [40, 70], BF16)
    assert bool((out[2:] == SENTINEL).all())


@pytest.mark.parametrize("n", [1, 40])
def test_paged_cache_elements_past_32_bits(n):
    HKV, D, ps, dt = 8, 128, 64, BF16
    pages = (1 << 32) // (ps * HKV * D) + 3
    kc = torch.zeros((pages, ps, HKV, D), device=DEV, dtype=dt)
    vc = torch.zeros((pages, ps, HKV, D), device=DEV, dtype=dt)
    g = gen(0)
    table = np.array([[pages - 1, 4, pages - 2]])
    kv = 2 * ps + 30
    for p in table[0]:
        kc[p], vc[p] = rand(g, ps, HKV, D, dt=dt), rand(g, ps, HKV, D, dt=dt)
    q = rand(g, n, 16, D, dt=dt)
    out = gdn.gdn_attention_paged(q, kc, vc, i32(table), i32([kv]), i32([0, n]), max_q=n)
    check_paged(out, q, kc, vc, table, [n], [kv], dt)


@pytest.mark.parametrize("dt,D,n", [(F32, 128, 1), (BF16, 128, 1), (BF16, 64, 5), (BF16, 256, 1), (BF16, 128, 200),
                                    (BF16, 256, 70)])
def test_paged_is_repeatable(dt, D, n):
    q, kc, vc, table = make_paged([n] * 3, [700 + n, 30 + n, 2000 + n], 8, 2, D, 16, dt)
    call = lambda: gdn.gdn_attention_paged(q, kc, vc, i32(table), i32([700 + n, 30 + n, 2000 + n]),
                                           i32([0, n, 2 * n, 3 * n]), max_q=n)
    a = call()
    for _ in range(3):
        assert torch.equal(a, call())


# ---------------------------------------------------------------- streams, graphs, refusals

def test_a_step_on_a_side_stream_and_in_a_graph():
    """plan -> norm and rotation with cache writes -> attention, on a stream of its own and as a
    captured graph: the same bits as on the default stream."""
    H, HKV, D, ps, B, M = 8, 2, 128, 16, 6, 12
    g = gen(4)
    P = 256
    a = np.arange(P)[:, None] * 10000.0 ** (-np.arange(D // 2) * 2.0 / D)[None, :]
    cos_sin = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).to(DEV)
    w = 1 + 0.1 * rand(g, D, dt=F32)
    cached = i32([3, 0, 40, 100, 15, 16])
    new, N = i32([1, 1, 1, 0, 1, 1]), 6
    pages = 100
    table = i32(np.arange(B * M).reshape(B, M))
    free = i32(np.arange(B * M, pages))
    qkv = rand(g, N, (H + 2 * HKV) * D)
    kc0, vc0 = rand(g, pages, ps, HKV, D), rand(g, pages, ps, HKV, D)
    ws = torch.empty(gdn.gdn_attention_paged_workspace_bytes(B, N, H, HKV, D, 1), dtype=torch.uint8, device=DEV)
    outs = torch.zeros(N, H, D, device=DEV, dtype=BF16)

    def step(kc, vc, t, out):
        o, kv, pos, slots, _, _ = gdn.gdn_page_plan(new, cached, t, free, page_size=ps, N=N, cursor=i32_zero)
        q, _ = gdn.gdn_qk_norm_rope(qkv, cos_sin, pos, H=H, HKV=HKV, D=D, q_weight=w, k_weight=w, slots=slots,
                                    k_cache=kc, v_cache=vc)
        gdn.gdn_attention_paged(q, kc, vc, t, kv, o, max_q=1, out=out, workspace=ws)

    i32_zero = i32([0])
    kc, vc, t = kc0.clone(), vc0.clone(), table.clone()
    step(kc, vc, t, outs)
    torch.cuda.synchronize()
    kc1, vc1, t1, out1 = kc0.clone(), vc0.clone(), table.clone(), torch.zeros_like(outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(kc1, vc1, t1, out1)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out1, outs) and torch.equal(kc1, kc) and torch.equal(t1, t)
    kc2, vc2, t2, out2 = kc0.clone(), vc0.clone(), table.clone(), torch.zeros_like(outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(kc2, vc2, t2, out2)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, outs) and torch.equal(kc2, kc) and torch.equal(vc2, vc) and torch.equal(t2, t)


def test_binding_refusals():
    g = gen(1)
    q, k, v = rand(g, 8, 4, 64), rand(g, 8, 2, 64), rand(g, 8, 2, 64)
    offs = i32([0, 8])
    call = gdn.gdn_attention_varlen
    for bad, status in ((lambda: call(q.cpu(), k, v, offs), 6), (lambda: call(q, k[:7], v, offs), 2),
                        (lambda: call(q, k.float(), v, offs), 2), (lambda: call(q.half(), k.half(), v.half(), offs), 5),
                        (lambda: call(q, k[:, :, ::2], v, offs), 2), (lambda: call(q, k, v, offs.long()), 2),
                        (lambda: call(q[:, :3], k, v, offs), 2),       # heads that do not divide
                        (lambda: call(q, k, v, offs, scale=float("nan")), 2),
                        (lambda: call(q.transpose(0, 1), k, v, offs), 2)):
        with pytest.raises(gdn.GdnError) as e:
            bad()
        assert e.value.status == status
    kc = rand(g, 3, 16, 2, 64)
    paged = lambda **kw: gdn.gdn_attention_paged(**{**dict(q=q, k_cache=kc, v_cache=kc, block_table=i32([[0, 1]]),
                                                           kv_lens=i32([20]), offsets=offs, max_q=8), **kw})
    paged()
    for kw, status in ((dict(v_cache=kc[:2]), 2), (dict(kv_lens=i32([1, 2])), 2), (dict(max_q=-1), 2),
                       (dict(workspace=torch.empty(256, dtype=torch.uint8, device=DEV)), 8),
                       (dict(k_cache=kc.float()), 2), (dict(offsets=i32([0, 4, 8])), 2)):
        with pytest.raises(gdn.GdnError) as e:
            paged(**kw)
        assert e.value.status == status
    with pytest.raises(gdn.GdnError):
        gdn.gdn_qk_norm_rope(rand(g, 4, 512), H=4, HKV=2, D=64, slots=i32([0, 1, 2, 3]))


def test_empty_calls():
    e = torch.empty
    out = gdn.gdn_attention_varlen(e(0, 4, 64, device=DEV, dtype=BF16), e(0, 2, 64, device=DEV, dtype=BF16),
                                   e(0, 2, 64, device=DEV, dtype=BF16), i32([0, 0]))
    assert out.shape == (0, 4, 64)
    q, k = gdn.gdn_qk_norm_rope(e(0, 512, device=DEV, dtype=BF16), H=4, HKV=2, D=64)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
