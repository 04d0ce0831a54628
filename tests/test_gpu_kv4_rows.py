"""Rows of 4-bit attention where it can go wrong: without keys, infinite, of extreme sizes, of malformed sequences."""
import pytest
import torch

import beam_ref
import serving_ref
import test_gpu_kv4 as kv4
import varlen_gated_delta_gb300 as gdn

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("size", [1e-36, 1e-30, 1e-22, 1e25, 1e36])
@pytest.mark.parametrize("n", [1, 20, 70])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_queries_and_scales_of_extreme_sizes(dtype, n, size):
    """Small factors with large queries, and the other way round, give ordinary scores."""
    p = kv4._problem(2, [n], [100], 4, 2, 64, 16, dtype)
    p["q"] = (p["q"].float() * size).to(dtype)
    scale = 0.3 / size
    kv4._check(p, kv4._run(p, scale=scale), scale)


@pytest.mark.parametrize("size", [1e-25, 1e25])
@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_head_scales_of_extreme_sizes(dtype, n, size):
    p = kv4._problem(3, [n], [100], 4, 2, 64, 16, dtype)
    p["q"] = (p["q"].float() * size).to(dtype)
    p["ts"][0] = torch.tensor([1.0 / size, 0.5 / size])
    kv4._check(p, kv4._run(p, scale=0.2), 0.2)


@pytest.mark.parametrize("size", [1e9, 1e20, 1e35])
@pytest.mark.parametrize("n,kv", [(1, 100), (20, 100), (70, 300), (40, 5000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scores_of_any_size_choose_one_key(dtype, n, kv, size):
    """With scores of 1e9 and more a row is the value of its best key."""
    p = kv4._problem(6, [n], [kv], 4, 2, 64, 16, dtype)
    p["q"] = (p["q"].float() * size).to(dtype)
    out = kv4._run(p).cpu().double()
    k, v = (serving_ref.cached_rows(beam_ref.kv4_values(c, 16, 64), p["table"][0], kv) for c in p["caches"])
    q, k, v = p["q"].double() / size, k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    x = torch.einsum("nhd,khd->nhk", q, k)
    x.masked_fill_(torch.ones(n, kv, dtype=torch.bool).triu(kv - n + 1)[:, None], -float("inf"))
    best = x.topk(2, -1)
    # a score is a sum of 64 products in fp32, each sum within 2^-23 of the largest: 2^-17 of sum |q k| covers it
    clear = best.values[..., 0] - best.values[..., 1] > 2.0 ** -16 * torch.einsum("nhd,khd->nhk", q.abs(), k.abs()).amax(-1)
    assert float(clear.float().mean()) > 0.9
    want = torch.gather(v.transpose(0, 1)[None].expand(n, -1, -1, -1), 2, best.indices[..., :1, None].expand(-1, -1, -1, 64))[:, :, 0]
    # the probability is a power of two: one rounding to the output's type, and one of the quotient
    tol = (torch.finfo(dtype).eps / 2 + 2.0 ** -23) * want.abs()
    assert bool(((out - want).abs() <= tol)[clear].all())


@pytest.mark.parametrize("factor", [2.0 ** -116, 2.0 ** 100])
@pytest.mark.parametrize("n,kv", [(1, 100), (1, 5000), (20, 100), (70, 300), (40, 5000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_value_scales_of_extreme_sizes(dtype, n, kv, factor):
    """A power of two as the values' scale moves the exponent of the outputs and nothing else."""
    p = kv4._problem(8, [n], [kv], 4, 2, 64, 16, dtype)
    want = kv4._run(p).double() * factor
    p["ts"][1] = torch.full((2,), factor)
    got = kv4._run(p).double()
    normal = want.abs() >= 2.0 ** -125
    assert float(normal.double().mean()) > 0.9 and torch.equal(got[normal], want[normal])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,kv", [(1, 90), (5, 90), (70, 90), (40, 5000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_infinite_queries_are_nan(dtype, n, kv, D):
    """Also where every score is -inf; a row that sees no key stays 0."""
    p = kv4._problem(n, [n, n], [kv, n - n // 2], 4, 2, D, 16, dtype)
    keys = p["caches"][0]
    keys[:, :, :16 * D // 2], keys[:, :, 16 * D // 2:] = 0x22, 0x38  # every key is a row of ones
    clean = kv4._run(p)
    odd = torch.zeros(clean.shape[:2], dtype=torch.bool, device="cuda")
    for row, h, d, x in ((0, 1, 3, "-inf"), (n - 1, 2, D - 1, "inf"), (2 * n - 1, 0, 0, "-inf")):
        p["q"][row, h, d] = float(x)
        odd[row, h] = True
    if n > 1:
        p["q"][n, 3, 1] = -float("inf")  # a row before the first key
    for scale in (0.0, -0.1):
        clean = kv4._run(dict(p, q=p["q"].nan_to_num(posinf=0, neginf=0)), scale=scale)
        out = kv4._run(p, scale=scale)
        assert bool(out[odd].isnan().all()) and torch.equal(out[~odd], clean[~odd])
        assert n == 1 or bool((out[n] == 0).all())


@pytest.mark.parametrize("n", [1, 24, 40])
def test_a_malformed_offset_leaves_the_others_alone(n):
    p = kv4._problem(5, [n, n, n], [40, 50, 60], 4, 2, 64, 16, BF16)
    out = torch.full(p["q"].shape, 3.0, dtype=BF16, device="cuda")
    kv4._run(dict(p, offsets=[0, -1, n, 2 * n]), out=out, max_q=n)  # the third sequence has rows n to 2 n
    alone = kv4._run(dict(p, q=p["q"][n:2 * n], table=p["table"][2:], kv=p["kv"][2:], offsets=[0, n]), max_q=n)
    assert torch.equal(out[n:2 * n], alone)
    assert bool((out[:n] == 3).all()) and bool((out[2 * n:] == 3).all())


@pytest.mark.parametrize("H,HKV,D", [(32, 8, 128), (8, 8, 64), (16, 4, 256)])
def test_hundreds_of_slices_without_keys(H, HKV, D):
    """Slices of sequences with no keys, or whose first rows see none, between ones that have some."""
    gen = torch.Generator().manual_seed(D)
    B = 400
    new = [int(x) for x in torch.randint(70, 90, (B,), generator=gen)]
    kv = [0 if b % 25 else new[b] + 60 for b in range(B)]
    kv[3], kv[200] = 5, 30  # fewer keys than rows
    p = kv4._problem(D, new, kv, H, HKV, D, 16, BF16)
    for _ in range(3):
        out = torch.full(p["q"].shape, 7.0, dtype=BF16, device="cuda")
        kv4._run(p, out=out)
        gdn.gdn_attention_status()
        for b in range(B):
            if kv[b] == 0:
                assert bool((out[p["offsets"][b]:p["offsets"][b + 1]] == 0).all())
    kv4._check(p, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_write_keeps_zeros_where_units_are_denormal(dtype):
    """Units below 2^-128, whose reciprocal leaves the range: zeros stay zeros, and values their nearest codes."""
    x = torch.zeros(1, 1, 32, dtype=dtype)
    x[0, 0, :3] = torch.tensor([2.0 ** -127, -2.0 ** -128, 2.0 ** -133])  # scale 2^-9, unit 2^-129
    x[0, 0, 16:18] = torch.tensor([2.0 ** -118, -2.0 ** -125])            # an ordinary group: scale 0.6875
    ts = torch.full((1,), 2.0 ** -120, device="cuda")
    cache = [torch.zeros(1, 1, gdn.kv4_page_bytes(16, 32), dtype=torch.uint8, device="cuda") for _ in "kv"]
    held, _ = gdn.gdn_kv4_write(x.cuda(), x.cuda(), torch.zeros(1, dtype=I32, device="cuda"), *cache, k_scale=ts, v_scale=ts, values=True)
    held = held.cpu().double()
    # 2^-127 and -2^-128 are 4 and -2 units, 2^-133 is nearest to none; of the other group 5.8 units and a 22nd of one
    assert held[0, 0, :16].tolist() == [2.0 ** -127, -2.0 ** -128] + [0.0] * 14
    assert held[0, 0, 16:].tolist() == [6 * 0.6875 * 2.0 ** -120] + [0.0] * 15


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [48, 64, 128, 256])
@pytest.mark.parametrize("M", [5, 400])
def test_slices_give_the_same_bits_every_time(M, D, dtype):
    """Short slices, a tile or two each, some without keys: what a CTA reads is not overwritten by its next item."""
    H, HKV, ps, pages = 32, 1, 32, 200
    new, kv = [67, 14, 83, 91, 128, 122, 94, 145, 79], [62, 14, 98, 91, 128, 0, 94, 145, 79]
    gen = torch.Generator(device="cuda").manual_seed(D)
    offsets = [0] + [sum(new[:i + 1]) for i in range(len(new))]
    # scales from 2^-9 to 240: mostly one key of a row counts, and a wrong value of it shows
    caches = [torch.randint(0, 120, (pages, HKV, gdn.kv4_page_bytes(ps, D)), dtype=torch.uint8, generator=gen, device="cuda") for _ in "kv"]
    table = torch.randint(0, pages, (len(new), M), dtype=I32, generator=gen, device="cuda")
    q = torch.randn(offsets[-1], H, D, generator=gen, device="cuda").to(dtype)
    a = (q, *caches, table, torch.tensor(kv, dtype=I32, device="cuda"), torch.tensor(offsets, dtype=I32, device="cuda"))
    want = gdn.gdn_attention_paged_kv4(*a, max_q=145)
    differs = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(300):
        differs |= (gdn.gdn_attention_paged_kv4(*a, max_q=145) != want).any()
    assert not bool(differs)
