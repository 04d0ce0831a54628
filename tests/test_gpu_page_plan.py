"""gdn_page_plan against a plain loop: integers, so every value must be equal."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import varlen_gated_delta_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from varlen_gated_delta_gb300 import build
    build.build()
    gdn.load_library()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _case(new, cached, ps, seed=0, spare=2, cursor=3, pad=0):
    rs = np.random.RandomState(seed)
    new, cached = [int(x) for x in new], [int(x) for x in cached]
    used = [-(-c // ps) for c in cached]
    need = [-(-(c + n) // ps) - u for n, c, u in zip(new, cached, used)]
    M = max(u + x for u, x in zip(used, need)) + spare
    M = max(M, 1)
    pool = rs.permutation(sum(used) + sum(need) + cursor + 4).tolist()
    table = np.full((len(new), M), -7)
    for b, u in enumerate(used):
        table[b, :u] = [pool.pop() for _ in range(u)]
    return dict(new=new, cached=cached, table=table, free=pool, ps=ps, cursor=cursor, N=sum(new) + pad)


def _run(c, **kw):
    t = i32(c["table"])
    got = gdn.gdn_page_plan(i32(c["new"]), i32(c["cached"]), t, i32(c["free"]), page_size=c["ps"],
                            N=c["N"], cursor=i32([c["cursor"]]), **kw)
    torch.cuda.synchronize()
    return [x.cpu().tolist() for x in got], t.cpu().tolist()


CASES = [
    ([1] * 64, list(range(0, 64 * 37, 37)), 64, 0),
    ([1], [0], 1, 0),
    ([0], [0], 16, 0),                                    # nothing at all
    ([0, 5, 0, 0, 3], [0, 16, 15, 17, 1], 16, 4),         # empty requests, page ends, unused tail
    ([16, 1, 15, 17], [0, 16, 16, 31], 16, 0),            # new tokens that end on and past page ends
    ([3000, 1, 70, 0, 129], [5, 6400, 63, 64, 0], 64, 0),  # several CTAs
    ([7] * 300, [11] * 300, 3, 100),                      # pages that are no power of two
]


@pytest.mark.parametrize("new,cached,ps,pad", CASES)
def test_plan_matches_a_loop(new, cached, ps, pad):
    c = _case(new, cached, ps, pad=pad)
    (offsets, kv, positions, slots, cursor, status), table = _run(c)
    want = ref.page_plan(c["new"], c["cached"], c["table"].tolist(), c["free"], ps, c["cursor"], c["N"])
    assert status == [0]
    assert (offsets, kv, positions, slots, table, cursor[0]) == want


@pytest.mark.parametrize("B", [8191, 8192])
def test_plan_of_as_many_requests_as_it_takes(B):
    rs = np.random.RandomState(B)
    c = _case(rs.randint(0, 5, B), rs.randint(0, 40, B), 16)
    (offsets, kv, positions, slots, cursor, status), table = _run(c)
    want = ref.page_plan(c["new"], c["cached"], c["table"].tolist(), c["free"], 16, c["cursor"], c["N"])
    assert status == [0]
    assert (offsets, kv, positions, slots, table, cursor[0]) == want


def test_lengths_and_cursor_carried_in_place_over_steps():
    ps, B, M = 4, 5, 20
    new, lens, cursor = i32([3, 0, 1, 9, 4]), i32([0] * B), i32([0])
    table, free = i32(np.full((B, M), -1)), i32(np.random.RandomState(1).permutation(80))
    want_table, want_lens, at = np.full((B, M), -1).tolist(), [0] * B, 0
    for step in range(4):
        got = gdn.gdn_page_plan(new, lens, table, free, page_size=ps, N=17, cursor=cursor,
                                kv_lens=lens, cursor_out=cursor)
        o, want_lens, p, s, want_table, at = ref.page_plan(new.tolist(), want_lens, want_table,
                                                           free.tolist(), ps, at, 17)
        assert got[1].data_ptr() == lens.data_ptr()
        assert lens.tolist() == want_lens and cursor.tolist() == [at] and table.tolist() == want_table
        assert got[0].tolist() == o and got[2].tolist() == p and got[3].tolist() == s
        new = i32([1] * B)


@pytest.mark.parametrize("over", ["cached", "new", "cursor", "none"])
def test_outputs_over_inputs_in_a_large_step(over):
    # many CTAs, every one of which reads the lengths and the cursor
    rs = np.random.RandomState(5)
    c = _case(rs.randint(0, 700, 200), rs.randint(0, 300, 200), 16, pad=9)
    new, cached, cursor, table = i32(c["new"]), i32(c["cached"]), i32([c["cursor"]]), i32(c["table"])
    out = {"cached": dict(kv_lens=cached), "new": dict(kv_lens=new), "cursor": dict(cursor_out=cursor), "none": {}}[over]
    got = gdn.gdn_page_plan(new, cached, table, i32(c["free"]), page_size=16, N=c["N"], cursor=cursor, **out)
    offsets, kv, positions, slots, at, status = [x.tolist() for x in got]
    want = ref.page_plan(c["new"], c["cached"], c["table"].tolist(), c["free"], 16, c["cursor"], c["N"])
    assert status == [0]
    assert (offsets, kv, positions, slots, table.tolist(), at[0]) == want


@pytest.mark.parametrize("what,status", [("negative", 2), ("negative cached", 2), ("cursor", 2), ("N", 4),
                                         ("free", 9), ("table", 9), ("overflow", 9)])
def test_a_step_that_cannot_be_planned_changes_nothing(what, status):
    c = _case([3, 40, 2], [10, 20, 30], 16, spare=0)
    if what == "negative":
        c["new"][1] = -1
    elif what == "negative cached":
        c["cached"][0] = -5
    elif what == "cursor":
        c["cursor"] = -1
    elif what == "N":
        c["N"] -= 1
    elif what == "free":
        c["cursor"] = len(c["free"]) - 1
    elif what == "table":
        c["cached"][1] = c["table"].shape[1] * 16 - 39
    else:
        c["cached"][1] = 2**31 - 10
    (offsets, kv, positions, slots, cursor, got), table = _run(c)
    assert got == [status]
    assert offsets == [0] * 4 and kv == c["cached"] and cursor == [c["cursor"]]
    assert positions == [0] * c["N"] and slots == [-1] * c["N"] and table == c["table"].tolist()
