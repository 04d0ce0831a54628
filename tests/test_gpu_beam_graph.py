"""A beam step captured into a CUDA graph, everything carried in place, against the same steps one by one."""
import pytest
import torch

import varlen_gated_delta_gb300 as gdn

pytestmark = pytest.mark.gpu
I32 = torch.int32


class Step:
    """Selection, states, tables and pages of G groups of K beams, from logits that are given."""

    def __init__(self, G, K, V, ps=16, M=12):
        gen = torch.Generator(device="cuda").manual_seed(3)
        B = G * K
        self.G, self.K, self.ps, self.pool = G, K, ps, B * M
        self.logits = torch.zeros(B, V, device="cuda", dtype=torch.bfloat16)
        self.scores = torch.zeros(G, K, device="cuda")
        self.finished = torch.zeros(G, K, dtype=torch.bool, device="cuda")
        self.tokens, self.parents = (torch.zeros(G, K, dtype=I32, device="cuda") for _ in range(2))
        self.states = [torch.randn(B, 3, 50, generator=gen, device="cuda"), torch.randn(B, 77, generator=gen, device="cuda").bfloat16()]
        self.caches = [torch.randn(self.pool, 5, generator=gen, device="cuda") for _ in range(2)]
        self.lens = torch.zeros(B, dtype=I32, device="cuda")
        self.table = torch.full((B, M), -1, dtype=I32, device="cuda")
        self.free = torch.arange(self.pool, dtype=I32, device="cuda")
        self.cursor, self.fork_status = torch.zeros(1, dtype=I32, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
        self.ones = torch.ones(B, dtype=I32, device="cuda")
        self.copies = torch.zeros(B, 2, dtype=I32, device="cuda")
        self.select_ws = torch.empty(gdn.gdn_beam_select_workspace_bytes(G, K, V, K), dtype=torch.uint8, device="cuda")
        self.fork_ws = torch.empty(gdn.gdn_page_fork_workspace_bytes(B, M, self.pool), dtype=torch.uint8, device="cuda")

    def run(self):
        gdn.gdn_page_plan(self.ones, self.lens, self.table, self.free, page_size=self.ps, N=self.G * self.K, cursor=self.cursor,
                          kv_lens=self.lens, cursor_out=self.cursor)
        gdn.gdn_beam_select(self.logits, self.scores, finished=self.finished, end_token=2, keep_rows=True, tokens=self.tokens,
                            parents=self.parents, scores_out=self.scores, finished_out=self.finished, workspace=self.select_ws)
        rows = self.parents.view(-1)
        gdn.gdn_state_reorder(self.states, rows)
        gdn.gdn_page_fork(rows, self.lens, self.table, self.free, page_size=self.ps, num_pages=self.pool, cursor=self.cursor,
                          table_out=self.table, kv_lens_out=self.lens, copies=self.copies, cursor_out=self.cursor,
                          status=self.fork_status, workspace=self.fork_ws)
        gdn.gdn_page_copy(self.caches, self.copies)

    def all(self):
        return [self.scores, self.finished, self.tokens, self.parents, *self.states, *self.caches, self.lens, self.table, self.free,
                self.cursor, self.fork_status]


def test_replayed_steps():
    a, b = Step(5, 4, 3001), Step(5, 4, 3001)
    saved = [t.clone() for t in b.all()]
    b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for t, s in zip(b.all(), saved):
        t.copy_(s)
    gen = torch.Generator(device="cuda").manual_seed(4)
    for _ in range(60):
        x = torch.randn(20, 3001, generator=gen, device="cuda").bfloat16()
        a.logits.copy_(x), b.logits.copy_(x)
        a.run()
        graph.replay()
        for s, t in zip(a.all(), b.all()):
            assert torch.equal(s, t)
        assert a.fork_status.item() == 0
    assert int(a.lens.min()) == int(a.lens.max()) == 60


def test_a_request_is_freed_and_its_pages_come_back():
    s = Step(3, 2, 100)
    for _ in range(40):
        s.run()
    used = int(s.cursor)
    rows = torch.tensor([0, 1, -1, -1, 4, 5], dtype=I32, device="cuda")
    mine = set(s.table[2:4][s.table[2:4] >= 0].tolist())
    others = set(s.table[[0, 1, 4, 5]].flatten().tolist()) - {-1}
    table, lens, copies, cursor, status = gdn.gdn_page_fork(rows, s.lens, s.table, s.free, page_size=s.ps, num_pages=s.pool, cursor=s.cursor)
    assert status.item() == 0 and bool((copies == -1).all()) and int(cursor) == used - len(mine - others)
    assert set(s.free[int(cursor):used].tolist()) == mine - others
    assert lens.tolist() == [40, 40, 0, 0, 40, 40] and bool((table[2:4] == -1).all())
