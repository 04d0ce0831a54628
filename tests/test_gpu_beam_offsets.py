"""Caches, logits and states whose places pass 32 bits: the calls give what they give on small ones with the same content."""
import pytest
import torch

import varlen_gated_delta_gb300 as gdn

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_4_bit_cache_of_more_than_4_gb(dtype):
    H, HKV, D, ps = 16, 8, 256, 64
    page = HKV * gdn.kv4_page_bytes(ps, D)
    pool = (1 << 32) // page + 40
    kv, new = [300, 1, 129], [1, 1, 1]
    # the rows' pages lie at both ends of the large cache, in the same order as in the small one
    used = [-(-n // ps) for n in kv]
    places = [pool - 1, 3, pool - 2, 0, pool - 17, pool - 30, 1, pool - 9, 2][:sum(used)]
    gen = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(sum(kv), HKV, D, generator=gen, device="cuda").to(dtype) for _ in "kv")
    q = torch.randn(40 * 3, H, D, generator=gen, device="cuda").to(dtype)
    results = []
    for pages, order in ((len(places), list(range(len(places)))), (pool, places)):
        kc, vc = (torch.empty(pages, HKV, gdn.kv4_page_bytes(ps, D), dtype=torch.uint8, device="cuda") for _ in "kv")
        table, slots, at = torch.full((3, max(used)), -1, dtype=I32), [], 0
        for b, n in enumerate(kv):
            table[b, :used[b]] = torch.tensor(order[at:at + used[b]])
            slots += [order[at + j // ps] * ps + j % ps for j in range(n)]
            at += used[b]
        held = gdn.gdn_kv4_write(k, v, _i32(slots), kc, vc, values=True)
        table = table.cuda()
        out = [gdn.gdn_attention_paged_kv4(q[:n * 3], kc, vc, table, _i32(kv), _i32([0, n, 2 * n, 3 * n]), max_q=n) for n in (1, 5, 40)]
        # a page copied from one end to the other, in both caches, and read there
        free = (pages - 3, 5) if pages == pool else None
        if free:
            gdn.gdn_page_copy([kc, vc], _i32([[order[0], free[1]], [order[1], free[0]]]))
            table[0, 0], table[0, 1] = free[1], free[0]
        out.append(gdn.gdn_attention_paged_kv4(q[:3], kc, vc, table, _i32(kv), _i32([0, 1, 2, 3]), max_q=1))
        results.append((*held, *out))
        del kc, vc
    for small, large in zip(*results):
        assert torch.equal(small, large)


def test_logits_of_more_than_2_31_values():
    rows, V, stride = 9, 5000, 1 << 28
    room = torch.empty((rows - 1) * stride + V, dtype=BF16, device="cuda")
    logits = room.as_strided((rows, V), (stride, 1))
    logits.copy_(torch.randn(rows, V, generator=torch.Generator().manual_seed(3)).to(BF16))
    scores = -torch.rand(3, 3, device="cuda")
    for a, b in zip(gdn.gdn_beam_select(logits, scores)[:3], gdn.gdn_beam_select(logits.contiguous(), scores)[:3]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("parents", [[0, 1, 1, 3, 3], [4, 3, 2, 2, 0]])  # whole rows copied; rows that change places
def test_states_of_more_than_4_gb(parents):
    state = torch.empty(5, (1 << 30) + 4096, dtype=torch.uint8, device="cuda")
    spots = [slice(0, 4096), slice(1 << 29, (1 << 29) + 4096), slice(1 << 30, None)]
    for i in range(5):
        for j, s in enumerate(spots):
            state[i, s] = 10 * i + j
    gdn.gdn_state_reorder([state], _i32(parents))
    for i, p in enumerate(parents):
        for j, s in enumerate(spots):
            assert bool((state[i, s] == 10 * p + j).all())
