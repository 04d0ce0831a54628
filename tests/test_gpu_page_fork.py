"""Forking, freeing, compacting and copying pages on the GPU, against lists on the CPU."""
import random

import pytest
import torch

import beam_ref
import varlen_gated_delta_gb300 as gdn

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _rows(rng, B, M, ps, pool, longest):
    """A sound state: rows that share full pages with an earlier one, or none.  (lens, rows, pages left over)."""
    left = list(range(pool))
    rng.shuffle(left)
    lens, rows = [], []
    for b in range(B):
        n = rng.choice([0, 1, ps, ps * M, rng.randint(0, longest), rng.randint(0, longest)])
        n = min(n, longest)
        common = []
        if rows and rng.random() < 0.6:
            other = rng.randrange(len(rows))
            common = rows[other][:rng.randint(0, lens[other] // ps)][:n // ps]
        need = -(-n // ps) - len(common)
        while need > len(left):
            n, common, need = 0, [], 0
        rows.append(common + [left.pop() for _ in range(need)])
        lens.append(n)
    return lens, rows, left


def _state(rng, B, M, ps, pool):
    lens, rows, left = _rows(rng, B, M, ps, pool, ps * M)
    live = sorted({x for r in rows for x in r})
    free = live + left  # the pages of the rows are handed out
    table = [r + [rng.choice([-1, 10 ** 6, 3]) for _ in range(M - len(r))] for r in rows]
    return lens, table, free, len(live)


FORKS = [(1, 1, 1, 1, 1), (4, 4, 5, 16, 40), (3, 8, 4, 3, 30), (64, 64, 20, 64, 900), (256, 100, 33, 16, 5001),
         (8192, 8192, 2, 16, 20000), (16, 16, 300, 1, 4000)]


@pytest.mark.parametrize("B,R,M,ps,pool,in_place", [(*f, False) for f in FORKS] + [(*f, True) for f in FORKS if f[0] == f[1]])
def test_fork(B, R, M, ps, pool, in_place):
    rng = random.Random(B * M + R)
    for kind in ("any", "few", "none", "same"):
        lens, table, free, cursor = _state(rng, B, M, ps, pool)
        some = [rng.randrange(B) for _ in range(3)]
        parents = [{"any": rng.randrange(-1, B), "few": rng.choice(some), "none": -1 - i, "same": i if i < B else -1}[kind] for i in range(R)]
        want = beam_ref.page_fork(parents, lens, table, free + [0] * R, cursor, ps)
        t, k, f, c = _i32(table), _i32(lens), _i32(free), _i32([cursor])
        kw = dict(table_out=t, kv_lens_out=k, cursor_out=c) if in_place else {}
        ws = torch.full((gdn.gdn_page_fork_workspace_bytes(B, M, pool),), 255, dtype=torch.uint8, device="cuda")
        to, ko, copies, co, status = gdn.gdn_page_fork(_i32(parents), k, t, f, page_size=ps, num_pages=pool, cursor=c, workspace=ws, **kw)
        if want[4] > len(free):
            assert status.item() == 9 and co.item() == cursor and f.tolist() == free and bool((copies == -1).all())
            assert to.tolist() == (table if in_place else [[-1] * M] * R) and ko.tolist() == (lens if in_place else [0] * R)
            continue
        rows, new_lens, pairs, new_free, new_cursor = want
        assert status.item() == 0 and co.item() == new_cursor and f.tolist() == new_free[:len(free)]
        assert ko.tolist() == new_lens
        assert to.tolist() == [r + [-1] * (M - len(r)) for r in rows]
        assert copies.tolist() == [list(p) for p in pairs] + [[-1, -1]] * (R - len(pairs))
        # what a table must keep: pages that are not full have one owner, and free pages none
        owners = {}
        for r, n in zip(rows, new_lens):
            if n % ps:
                owners[r[-1]] = owners.get(r[-1], 0) + sum(r[-1] in x for x in rows)
        assert all(v == 1 for v in owners.values())
        assert not set(new_free[new_cursor:len(free)]) & {x for r in rows for x in r}


def test_fork_takes_and_refuses():
    # two children of a row with a page and a half; nothing to hand out
    t, k, c = _i32([[5, 6, 0]]), _i32([24]), _i32([2])
    for free, status in (([5, 6], 9), ([5, 6, 4], 0)):
        got = gdn.gdn_page_fork(_i32([0, 0]), k, t, _i32(free), page_size=16, num_pages=8, cursor=c)
        assert got[4].item() == status
    assert got[0].tolist() == [[5, 6, -1], [5, 4, -1]] and got[2].tolist() == [[6, 4], [-1, -1]] and got[3].item() == 3
    # out of range: a parent, a length, a page, the cursor; and more pages than were handed out
    for bad in (dict(parents=[1]), dict(lens=[-1]), dict(lens=[49]), dict(table=[[5, 8, 0]]), dict(table=[[-1, 6, 0]]), dict(cursor=-1),
                dict(cursor=1, parents=[-1])):
        a = dict(dict(parents=[0], lens=[24], table=[[5, 6, 0]], cursor=2), **bad)
        free = _i32([5, 6, 4])
        to, ko, copies, co, status = gdn.gdn_page_fork(_i32(a["parents"]), _i32(a["lens"]), _i32(a["table"]), free, page_size=16, num_pages=8,
                                                       cursor=_i32([a["cursor"]]))
        assert status.item() == 2 and co.item() == a["cursor"] and free.tolist() == [5, 6, 4]
        assert to.tolist() == [[-1, -1, -1]] and ko.tolist() == [0] and copies.tolist() == [[-1, -1]]
    for bad in (dict(parents=_i32([[0]])), dict(kv_lens=_i32([1, 2])), dict(block_table=t.long()), dict(cursor=_i32([1, 2])),
                dict(table_out=t, parents=_i32([0, 0])), dict(page_size=0), dict(num_pages=0),
                dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_page_fork(**dict(dict(parents=_i32([0]), kv_lens=k, block_table=t, free_pages=_i32([1]), page_size=16, num_pages=8,
                                          cursor=c), **bad))


@pytest.mark.parametrize("cursor", [4, 5, 1 << 30])
def test_fork_refuses_a_cursor_past_the_list(cursor):
    # (pages that go back would be put past its end: words behind the list keep their values)
    room = _i32([5, 6, 4, 77, 77, 77])
    free = room[:3]
    to, ko, copies, co, status = gdn.gdn_page_fork(_i32([-1]), _i32([24]), _i32([[5, 6, 0]]), free, page_size=16, num_pages=8,
                                                   cursor=_i32([cursor]))
    assert status.item() == 2 and co.item() == cursor and room.tolist() == [5, 6, 4, 77, 77, 77]
    assert to.tolist() == [[-1, -1, -1]] and ko.tolist() == [0] and copies.tolist() == [[-1, -1]]


@pytest.mark.parametrize("B,M,ps,pool", [(1, 1, 1, 1), (1, 2, 16, 2), (4, 5, 16, 40), (64, 20, 64, 900), (300, 33, 16, 7777), (2, 1, 16, 100000),
                                         (9000 - 900, 1, 4, 9000), (16, 2000, 1, 33000)])
def test_compact(B, M, ps, pool):
    rng = random.Random(B + M)
    for full in (False, True):
        lens, table, free, live = _state(rng, B, M, ps, pool)
        if full and live > 1:  # no gaps
            to = {p: i for i, p in enumerate(free)}
            table = [[to.get(p, p) if j < -(-n // ps) else p for j, p in enumerate(r)] for r, n in zip(table, lens)]
        rows, pairs, n = beam_ref.page_compact(lens, table, ps)
        t, k = _i32(table), _i32(lens)
        for in_place in (False, True):
            ws = torch.full((gdn.gdn_page_compact_workspace_bytes(pool),), 255, dtype=torch.uint8, device="cuda")
            to, copies, fp, cursor, status = gdn.gdn_page_compact(k, t, page_size=ps, num_pages=pool, workspace=ws,
                                                                  table_out=t if in_place else None)
            assert status.item() == 0 and cursor.item() == n and fp.tolist() == list(range(pool))
            assert to.tolist() == [r + [-1] * (M - len(r)) for r in rows]
            assert copies.tolist() == [list(p) for p in pairs] + [[-1, -1]] * (pool // 2 - len(pairs))


def test_compact_refuses():
    for lens, table in (([33], [[1, 2]]), ([-1], [[1, 2]]), ([20], [[1, 9]]), ([20], [[-1, 1]])):
        t, free, cursor = _i32(table), _i32([7] * 9), _i32([5])
        to, copies, _, _, status = gdn.gdn_page_compact(_i32(lens), t, page_size=16, num_pages=9, free_pages=free, cursor_out=cursor)
        assert status.item() == 2 and to.tolist() == [[-1, -1]] and bool((copies == -1).all())
        assert free.tolist() == [7] * 9 and cursor.item() == 5
    with pytest.raises(gdn.GdnError):
        gdn.gdn_page_compact(_i32([1]), _i32([[0]]), page_size=16, num_pages=0)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_page_compact(_i32([1, 1]), _i32([[0]]), page_size=16, num_pages=4)


@pytest.mark.parametrize("shape,dtype", [((64, 8, 128), torch.bfloat16), ((3,), torch.uint8), ((5, 7), torch.float32), ((1,), torch.bfloat16),
                                         ((40000,), torch.float32), ((0, 4), torch.float32)])
def test_copy(shape, dtype):
    gen = torch.Generator(device="cuda").manual_seed(1)
    pool = 50
    caches = [torch.randint(0, 100, (pool, *shape), generator=gen, device="cuda").to(dtype) for _ in range(3)]
    order = torch.randperm(pool, generator=gen, device="cuda").to(I32)
    pairs = torch.stack([order[:20], order[20:40]], 1)
    pairs[3] = torch.tensor([1, pool])  # outside: skipped
    pairs[4, 0] = pool + 7
    pairs[5, 1] = -3
    pairs = torch.cat([pairs, torch.full((400, 2), -1, dtype=I32, device="cuda"), order[40:42].view(1, 2)])
    want = [c.clone() for c in caches]
    for i, (a, b) in enumerate(pairs.tolist()):
        if i not in (3, 4, 5) and a >= 0:
            for c, w in zip(caches, want):
                w[b] = c[a]
    gdn.gdn_page_copy(caches, pairs)
    for c, w in zip(caches, want):
        assert torch.equal(c, w)


def test_copy_refusals_and_nothing_to_do():
    cache, pairs = torch.zeros(4, 8, device="cuda"), _i32([[0, 1]])
    for caches, p in (([cache[:, :3]], pairs), ([cache, cache[:3]], pairs), ([cache], pairs.long()), ([cache], pairs.view(2)),
                      ([cache], pairs.cpu()), ([cache] * 129, pairs), ([cache], _i32([[0, 1, 2]]))):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_page_copy(caches, p)
    gdn.gdn_page_copy([], pairs)
    gdn.gdn_page_copy([cache], pairs[:0])
    gdn.gdn_page_copy([cache[:0]], pairs)
