"""4-bit caches on the GPU against their definition in 64 bits: the write bit for bit, attention within its roundings."""
import math

import pytest
import torch

import beam_ref
import serving_ref
import varlen_gated_delta_gb300 as gdn

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _rand(gen, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


# ---------------------------------------------------------------- write

def _expected_write(x, ts, slots, cache, ps):
    N, H, D = x.shape
    cache, held = cache.clone(), torch.zeros(N, H, D)
    scales = torch.ones(H) if ts is None else ts
    for n in range(N):
        for h in range(H):
            for g in range(D // 16):
                codes, byte, values = beam_ref.kv4_group(x[n, h, 16 * g:16 * g + 16].float().tolist(), float(scales[h]))
                held[n, h, 16 * g:16 * g + 16] = torch.tensor(values, dtype=torch.float64).float()
                slot = int(slots[n])
                if 0 <= slot < cache.shape[0] * ps:
                    page, at = divmod(slot, ps)
                    for i in range(8):
                        cache[page, h, at * D // 2 + 8 * g + i] = codes[2 * i] | codes[2 * i + 1] << 4
                    cache[page, h, ps * D // 2 + at * D // 16 + g] = byte
    return cache, held.to(x.dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,H,D,ps,scaled,strided", [
    (1, 1, 16, 16, False, False), (5, 2, 64, 16, True, False), (3, 3, 80, 48, True, True), (17, 2, 128, 64, False, True),
    (2, 1, 256, 32, True, False)])
def test_write(dtype, N, H, D, ps, scaled, strided):
    gen = torch.Generator().manual_seed(N * D)
    pages = -(-N // ps) + 2
    rows = _rand(gen, N, 2 * H * D + (3 if strided else 0), dtype=dtype)
    rows[0, :4] = torch.tensor([0.0, -0.0, 1e-8, -1e-8])
    rows[N - 1, H * D:H * D + 16] = 0  # a group of nothing
    k, v = (rows[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(2))
    ts = (torch.rand(H, generator=gen) * 0.2 + 0.01) if scaled else None
    slots = torch.randperm(pages * ps, generator=gen)[:N].to(I32)
    if N > 2:
        slots[1], slots[2] = -1, pages * ps  # nowhere
    empty = torch.randint(0, 256, (pages, H, ps * D * 9 // 16), generator=gen, dtype=torch.uint8)
    cache = [empty.clone().cuda(), empty.clone().cuda()]
    dev = rows.cuda()
    dk, dv = (dev[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(2))
    scale = None if ts is None else ts.cuda()
    ko, vo = gdn.gdn_kv4_write(dk, dv, slots.cuda(), *cache, k_scale=scale, v_scale=scale, values=True)
    for x, got, held in ((k, cache[0], ko), (v, cache[1], vo)):
        want, values = _expected_write(x, ts, slots, empty, ps)
        assert torch.equal(got.cpu(), want)
        assert torch.equal(held.cpu(), values)
    again = [empty.clone().cuda(), empty.clone().cuda()]
    assert gdn.gdn_kv4_write(dk, dv, slots.cuda(), *again, k_scale=scale, v_scale=scale) == (None, None)
    assert torch.equal(again[0], cache[0]) and torch.equal(again[1], cache[1])


def test_write_of_every_halfway_value_and_of_what_is_not_finite():
    """Halfway between codes in units of a scale of 1 (the group's largest is 6), and infinities, NaN and tiny groups."""
    half = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    rows = [half + [-x for x in half] + [6.0, -6.0], [x * 1.0078125 for x in half] + [x * 0.9921875 for x in half] + [6.0, 0.5],
            [float("inf"), -float("inf")] + [1.0] * 14, [float("nan")] + [3.0] * 15, [float("nan")] * 16, [1e-30] * 16, [0.0] * 16,
            [1e4] * 16, [2.0 ** -9 * 3] * 16]
    x = torch.tensor(rows, dtype=F32).view(1, 1, 16 * len(rows))[..., :144].contiguous()
    for dtype in (BF16, F32):
        k = x.to(dtype)
        cache = torch.zeros(1, 1, 16 * 144 * 9 // 16, dtype=torch.uint8)
        c, d = cache.cuda(), cache.cuda()
        held, _ = gdn.gdn_kv4_write(k.cuda(), k.cuda(), _i32([3]), c, d, values=True)
        want, values = _expected_write(k, None, [3], cache, 16)
        assert torch.equal(c.cpu(), want) and torch.equal(d.cpu(), want)
        assert torch.equal(held.cpu(), values)


def test_write_refusals():
    k = torch.zeros(2, 2, 64, device="cuda", dtype=BF16)
    cache = torch.zeros(3, 2, 16 * 36, dtype=torch.uint8, device="cuda")
    slots = _i32([0, 1])
    for bad in (dict(k=k[:, :, :60]), dict(k=k.half(), v=k.half()), dict(v=k[:1]), dict(slots=slots[:1]), dict(slots=slots.long()),
                dict(k_cache=cache[:, :1]), dict(k_cache=cache[:, :, 1:]), dict(v_cache=cache[:, :, :288].contiguous()),
                dict(k_scale=torch.ones(3, device="cuda")), dict(k_cache=cache.cpu()), dict(k_cache=cache.char()),
                dict(k_cache=cache[:, :, :288].contiguous(), v_cache=cache[:, :, :288].contiguous())):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_kv4_write(**dict(dict(k=k, v=k, slots=slots, k_cache=cache, v_cache=cache.clone()), **bad))
    gdn.gdn_kv4_write(k[:0], k[:0], slots[:0], cache, cache.clone(), values=True)


# ---------------------------------------------------------------- attention

def _problem(seed, new, kv, H, HKV, D, ps, dtype, scaled=False, spare=3, extra=0, max_pages=None):
    gen = torch.Generator().manual_seed(seed)
    used = [-(-k // ps) for k in kv]
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=gen)
    M = max_pages or max(1, max(used))
    table, at = torch.full((len(kv), M), -1, dtype=I32), 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    ts = [torch.rand(HKV, generator=gen) * 0.3 + 0.02 if scaled else None for _ in "kv"]
    caches = [beam_ref.kv4_cache(_rand(gen, pages, HKV, ps, D, dtype=F32), t) for t in ts]
    # what no sequence holds may be anything
    for cache in caches:
        for b, (u, k) in enumerate(zip(used, kv)):
            if k % ps:
                page = int(table[b, u - 1])
                cache[page, :, :ps * D // 2].view(HKV, ps, -1)[:, k % ps:] = 255
                cache[page, :, ps * D // 2:].view(HKV, ps, -1)[:, k % ps:] = 255
        cache[order[at:]] = 255
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    q = _rand(gen, offsets[-1] + extra, H, D, dtype=dtype, std=1.5)
    return dict(q=q, caches=caches, table=table, kv=list(kv), offsets=offsets, ps=ps, ts=ts)


def _run(p, **kw):
    ks, vs = (None if t is None else t.cuda() for t in p["ts"])
    a = dict(max_q=max(b - a for a, b in zip(p["offsets"], p["offsets"][1:])), k_scale=ks, v_scale=vs)
    a.update(kw)
    return gdn.gdn_attention_paged_kv4(p["q"].cuda(), p["caches"][0].cuda(), p["caches"][1].cuda(), p["table"].cuda(), _i32(p["kv"]),
                                       _i32(p["offsets"]), **a)


def _check(p, out, scale=None):
    q, ps, D = p["q"], p["ps"], p["q"].shape[2]
    k, v = (beam_ref.kv4_values(c, ps, D, t) for c, t in zip(p["caches"], p["ts"]))
    half = torch.finfo(q.dtype).eps / 2
    for b, kv in enumerate(p["kv"]):
        rows = slice(p["offsets"][b], p["offsets"][b + 1])
        kb, vb = (serving_ref.cached_rows(x, p["table"][b], kv) for x in (k, v))
        want, mag = serving_ref.attention(q[rows], kb, vb, scale)
        # A score is a sum of D products in fp32 (and of an fp32 query's two parts): with its factor at most `far` off, in nats,
        # where the tensor cores may truncate each addition (2^-23).  That moves p by the same relative amount, in
        # the numerator and the sum; 2^-21: the exponential and the sums over keys.  bf16: p is rounded to 11 bits (2^-12).
        size = (q[rows].double().abs().amax() * kb.abs().sum(-1).amax() if want.numel() and kv else torch.tensor(0.0)) * abs(scale or 1 / math.sqrt(D))
        far = 2 * float(size) * (D + 8) * 2.0 ** -23
        # p is held 2^14 times as large in fp16, whose values below 2^-14 lie 2^-24 apart: a p of less than 2^-28 of the row's
        # largest is off by up to 2^-25 / 2^14 of it, and the sum is at least that largest: |v_j| 2^-39 for each key.
        lost = vb.abs().sum(0).repeat_interleave(q.shape[1] // max(1, vb.shape[1]), 0) * 2.0 ** -39 if kv else 0.0
        tol = half * want.abs() + lost + (2 * far + 2.0 ** -21 + kv * 2.0 ** -24 + (2.0 ** -12 if q.dtype == BF16 else 2.0 ** -21)) * mag + 1e-30
        got = out[rows].cpu().double()
        worst = ((got - want).abs() / tol).max() if got.numel() else 0.0
        assert worst <= 1, f"sequence {b}: {float(worst):.2f} of the tolerance"


HEADS = [(4, 4, 64), (8, 2, 128), (8, 1, 128), (32, 2, 64), (6, 2, 80), (3, 1, 96), (4, 2, 256), (16, 2, 256), (2, 2, 16), (66, 1, 32)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,HKV,D", HEADS)
def test_single_tokens(H, HKV, D, dtype):
    p = _problem(H * D, [1] * 6, [1, 15, 16, 64, 129, 700], H, HKV, D, 16 if D < 128 else 64, dtype, scaled=H % 3 == 0)
    _check(p, _run(p))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,HKV,D", HEADS)
def test_drafts_and_slices(H, HKV, D, dtype):
    new = [3, 1, 17, 0, 5, 70]
    p = _problem(H + D, new, [3, 40, 17, 9, 333, 190], H, HKV, D, 48 if D > 64 else 32, dtype, scaled=H % 2 == 0, extra=2)
    _check(p, _run(p))


@pytest.mark.parametrize("ps", [16, 32, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 9])
def test_page_sizes(ps, n):
    p = _problem(ps + n, [n, n], [ps * 2 + 5 + n, 301], 8, 2, 128, ps, BF16)
    _check(p, _run(p))


@pytest.mark.parametrize("new", [[1], [0, 1, 3], [1, 1, 1, 70], [20, 16, 17]])
def test_more_sequences_than_threads(new):
    rng = torch.Generator().manual_seed(len(new))
    new = [new[i % len(new)] for i in range(300)]
    kv = [n + int(k) for n, k in zip(new, torch.randint(0, 150, (300,), generator=rng))]
    p = _problem(8, new, kv, 4, 2, 64, 16, BF16)
    _check(p, _run(p))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 4, 40])
def test_long_histories_split_over_ctas(n, dtype):
    p = _problem(n, [n], [9001], 8, 2, 128, 64, dtype, scaled=True)
    _check(p, _run(p))


@pytest.mark.parametrize("n", [1, 5, 130])
def test_rows_without_keys_and_rows_behind_the_last_sequence(n):
    p = _problem(n, [n, n, n], [n, 0, max(0, n - 2)], 4, 2, 64, 16, BF16, extra=3)
    out = torch.full(p["q"].shape, 7.0, dtype=BF16, device="cuda")
    got = _run(p, out=out)
    assert got is out
    _check(p, out)
    assert bool((out[n:2 * n] == 0).all()) and bool((out[3 * n:] == 7).all())


@pytest.mark.parametrize("scale", [0.03, -0.2, 1e-25, 3.0])
def test_scales(scale):
    p = _problem(1, [1, 20], [50, 77], 4, 2, 64, 16, BF16, scaled=True)
    _check(p, _run(p, scale=scale), scale)


@pytest.mark.parametrize("size", [1e-20, 1e-6, 1e12])
@pytest.mark.parametrize("n", [1, 20])
def test_queries_of_any_size(size, n):
    """Rows are scaled by powers of two: small and large queries keep their precision."""
    p = _problem(2, [n], [100], 4, 2, 64, 16, F32)
    p["q"] = p["q"] * size
    scale = 0.3 / size
    _check(p, _run(p, scale=scale), scale)


@pytest.mark.parametrize("n", [1, 12, 200])
def test_pages_outside_the_cache_read_as_zeros(n):
    p = _problem(3, [n, n], [210, 250], 8, 2, 64, 16, BF16)
    p["table"][0, 2], p["table"][0, 5], p["table"][1, 0] = -1, p["caches"][0].shape[0], 1 << 30
    _check(p, _run(p))


@pytest.mark.parametrize("n", [1, 40])
def test_non_finite_queries_stay_in_their_rows(n):
    p = _problem(4, [n, n], [90, 60], 4, 2, 64, 16, BF16)
    clean = _run(p)
    p["q"][0, 1, 3], p["q"][n, 2, 0] = float("nan"), float("inf")
    out = _run(p)
    odd = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    odd[0, 1] = odd[n, 2] = True
    assert bool(out[odd].isnan().all()) and torch.equal(out[~odd], clean[~odd])


@pytest.mark.parametrize("n", [1, 24])
def test_malformed_sequences_are_left_out(n):
    p = _problem(5, [n, n, n], [40, 50, 60], 4, 2, 64, 16, BF16)
    want = _run(p)
    for kv in (-1, 65 * 16, 1 << 30):
        out = torch.full_like(want, 3.0)
        _run(dict(p, kv=[40, kv, 60]), out=out)
        assert torch.equal(out[:n], want[:n]) and torch.equal(out[2 * n:], want[2 * n:]) and bool((out[n:2 * n] == 3).all())
    out = torch.full_like(want, 3.0)
    if n > 1:  # more rows than max_q
        _run(dict(p, offsets=[0, n, 3 * n - 1, 3 * n]), out=out, max_q=n)
        assert torch.equal(out[:n], want[:n]) and bool((out[n:3 * n - 1] == 3).all())
    out.fill_(3.0)
    _run(dict(p, offsets=[0, -1, n, 2 * n]), out=out, max_q=n)
    assert bool((out[n + 1:] != 3).any()) or n == 1


@pytest.mark.parametrize("n", [1, 5, 40])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_queries_off_16_byte_boundaries(dtype, n):
    """Rows that begin at any element take the scalar loads."""
    p = _problem(9, [n, n], [50, 120], 8, 2, 96, 16, dtype)
    want = _run(p)
    for first in (1, 3):
        room = torch.zeros(2 * n, 8 * 96 + 5, dtype=dtype, device="cuda")
        view = room[:, first:first + 8 * 96].unflatten(1, (8, 96))
        view.copy_(p["q"])
        got = gdn.gdn_attention_paged_kv4(view, p["caches"][0].cuda(), p["caches"][1].cuda(), p["table"].cuda(), _i32(p["kv"]),
                                          _i32(p["offsets"]), max_q=n)
        assert torch.equal(got, want)


def test_another_stream_and_thread_of_work():
    """Two calls at once, each on its own stream with a workspace of its own."""
    p = _problem(10, [1, 30, 4], [900, 700, 65], 8, 2, 128, 64, BF16)
    want = _run(p)
    a = [x.cuda() for x in (p["q"], *p["caches"], p["table"])] + [_i32(p["kv"]), _i32(p["offsets"])]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(gdn.gdn_attention_paged_kv4(*a, max_q=30))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_strided_queries_and_workspace():
    p = _problem(6, [1, 30], [80, 99], 4, 2, 64, 16, BF16)
    want = _run(p)
    wide = torch.zeros(31, 6, 64, dtype=BF16, device="cuda")
    wide[:, 1:5] = p["q"].cuda()
    need = gdn.gdn_attention_paged_kv4_workspace_bytes(2, 31, 4, 2, 64, 30)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = gdn.gdn_attention_paged_kv4(wide[:, 1:5], p["caches"][0].cuda(), p["caches"][1].cuda(), p["table"].cuda(), _i32(p["kv"]),
                                      _i32(p["offsets"]), max_q=30, workspace=ws)
    assert torch.equal(out, want)
    with pytest.raises(gdn.GdnError):
        _run(p, workspace=ws[:256])


@pytest.mark.parametrize("n", [1, 6, 30])
def test_reruns_and_graphs_give_the_same_bits(n):
    p = _problem(7, [n] * 9, [700, 3000, 1, 50, 64, 65, 900, 128, 2000][:9] if n == 1 else [700, 3000, 50, 50, 64, 65, 900, 128, 2000],
                 8, 2, 128, 64, BF16)
    a = [x.cuda() for x in (p["q"], *p["caches"], p["table"])] + [_i32(p["kv"]), _i32(p["offsets"])]
    want = gdn.gdn_attention_paged_kv4(*a, max_q=n)
    _check(p, want)
    out = torch.zeros_like(want)
    ws = torch.empty(gdn.gdn_attention_paged_kv4_workspace_bytes(9, 9 * n, 8, 2, 128, n), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        gdn.gdn_attention_paged_kv4(*a, max_q=n, out=out, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gdn.gdn_attention_paged_kv4(*a, max_q=n, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    a[4].copy_(_i32([x - 1 for x in p["kv"]]) if n == 1 else a[4])  # other lengths, the same graph
    graph.replay()
    assert torch.equal(out, gdn.gdn_attention_paged_kv4(*a, max_q=n))
    assert n > 1 or bool((out[2] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 40])
def test_nothing_past_the_workspace_and_the_rows(n, D, dtype):
    """Every CTA has parts of two sequences to leave; the words behind the workspace and the output keep their values."""
    H, HKV, ps, pages, B = 8, 1, 64, 2000, 7
    gen = torch.Generator(device="cuda").manual_seed(D)
    cache = torch.randint(0, 120, (pages, HKV, gdn.kv4_page_bytes(ps, D)), dtype=torch.uint8, generator=gen, device="cuda")
    table = torch.randint(0, pages, (B, 500), dtype=I32, generator=gen, device="cuda")
    kv = _i32([31000 - 1700 * b for b in range(B)])
    q = torch.randn(B * n, H, D, generator=gen, device="cuda").to(dtype)
    need = gdn.gdn_attention_paged_kv4_workspace_bytes(B, B * n, H, HKV, D, n)
    room = torch.full((need + 65536,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((B * n + 5, H, D), 3.0, dtype=dtype, device="cuda")
    gdn.gdn_attention_paged_kv4(q, cache, cache, table, kv, _i32([n * b for b in range(B + 1)]), max_q=n, workspace=room[:need],
                                out=out[:B * n])
    assert bool((room[need:] == 77).all()) and bool((out[B * n:] == 3.0).all())
    want = gdn.gdn_attention_paged_kv4(q, cache, cache, table, kv, _i32([n * b for b in range(B + 1)]), max_q=n)
    assert torch.equal(out[:B * n], want) and bool(torch.isfinite(want).all())
