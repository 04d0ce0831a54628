"""Beam search with a small stack of a gated-delta and a softmax-attention layer, its cache held in 4 bits.

Each request has `beams` rows.  A prompt runs once for a request and is then forked to its beams; after that, per step:

  gdn_page_plan              pages, slots and positions of the new tokens
  delta layer                gdn_layer_varlen, conv and delta states carried in place
  attention layer            gdn_qk_norm_rope, gdn_kv4_write, gdn_attention_paged_kv4
  gdn_beam_select            the best continuations of each request; beams that go on keep their rows
  gdn_state_reorder          conv and delta states follow them
  gdn_page_fork, _page_copy  so do the block tables: full pages are shared, a page that is still written is copied

Weights are random.  At the end every beam's tokens are run again by themselves, and the scores of both ways are compared.

  python examples/beam_serving.py [--requests 3] [--beams 4] [--longest 90] [--steps 24]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import varlen_gated_delta_gb300 as gdn  # noqa: E402

F32, I32 = torch.float32, torch.int32


class BeamStack:
    """One gated-delta layer and one attention layer for `rows` rows of tokens."""

    def __init__(self, rows, max_tokens, vocab=500, width=256, HQ=2, H=4, AH=4, AHKV=2, D=64, page_size=16, device="cuda",
                 seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rand = lambda *s, std=1.0: torch.randn(*s, generator=g, device=device) * std
        lin = lambda i, o: rand(i, o, std=1 / math.sqrt(i))
        self.dev, self.B, self.width, self.ps, self.vocab = device, rows, width, page_size, vocab
        self.HQ, self.H, self.AH, self.AHKV, self.D = HQ, H, AH, AHKV, D
        W = 2 * HQ * D + H * D
        self.embed, self.head = rand(vocab, width), lin(width, vocab) * 4
        self.delta = dict(qkv=lin(width, W), gates=lin(width, 2 * H), out=lin(H * D, width), conv=rand(W, 4, std=0.5),
                          A_log=torch.rand(H, generator=g, device=device) * math.log(16.0), dt_bias=rand(H))
        self.attn = dict(qkv=lin(width, (AH + 2 * AHKV) * D), out=lin(AH * D, width), qw=1 + 0.1 * rand(D), kw=1 + 0.1 * rand(D))
        angle = (torch.arange(max_tokens, dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)[None, :])
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)
        self.max_pages = -(-max_tokens // page_size)
        self.pages = rows * self.max_pages
        self.reset()

    def reset(self):
        """Empty states, cache and page tables."""
        B, dev = self.B, self.dev
        self.conv_state = torch.zeros(B, self.delta["conv"].shape[0], 3, device=dev)
        self.state = torch.zeros(B, self.H, self.D, self.D, device=dev)
        self.k, self.v = (torch.zeros(self.pages, self.AHKV, gdn.kv4_page_bytes(self.ps, self.D), dtype=torch.uint8, device=dev)
                          for _ in "kv")
        self.lens = torch.zeros(B, dtype=I32, device=dev)
        self.table = torch.full((B, self.max_pages), -1, dtype=I32, device=dev)
        self.free = torch.arange(self.pages, dtype=I32, device=dev)
        self.cursor = torch.zeros(1, dtype=I32, device=dev)
        self.status = torch.zeros(1, dtype=I32, device=dev)

    def step(self, tokens, new_lens, longest):
        """Logits of every token of a packed batch."""
        N, H, HQ, D, AH, AHKV = tokens.numel(), self.H, self.HQ, self.D, self.AH, self.AHKV
        offsets, _, positions, slots, _, status = gdn.gdn_page_plan(
            new_lens, self.lens, self.table, self.free, page_size=self.ps, N=N, cursor=self.cursor, kv_lens=self.lens,
            cursor_out=self.cursor)
        self.status = torch.maximum(self.status, status)
        norm = lambda x: torch.nn.functional.rms_norm(x, (self.width,))
        x = self.embed[tokens.long()]
        L, h = self.delta, norm(x)
        a, b = (h @ L["gates"]).split(H, 1)
        y, _, _ = gdn.gdn_layer_varlen(
            h @ L["qkv"], L["conv"], None, a.contiguous(), b.contiguous(), L["A_log"], L["dt_bias"], offsets, self.conv_state,
            self.state, H=H, HQ=HQ, K=D, V=D, conv_fin=self.conv_state, state_fin=self.state)
        x = x + y.reshape(N, -1) @ L["out"]
        L = self.attn
        qkv = norm(x) @ L["qkv"]
        q, k = gdn.gdn_qk_norm_rope(qkv, self.cos_sin, positions, H=AH, HKV=AHKV, D=D, q_weight=L["qw"], k_weight=L["kw"])
        gdn.gdn_kv4_write(k, qkv[:, (AH + AHKV) * D:].view(N, AHKV, D), slots, self.k, self.v)
        y = gdn.gdn_attention_paged_kv4(q, self.k, self.v, self.table, self.lens, offsets, max_q=longest)
        x = x + y.reshape(N, -1) @ L["out"]
        return norm(x) @ self.head

    def follow(self, parents):
        """States, block tables and pages of each row continue those of row parents[row]."""
        gdn.gdn_state_reorder([self.conv_state, self.state], parents)
        _, _, copies, _, status = gdn.gdn_page_fork(
            parents, self.lens, self.table, self.free, page_size=self.ps, num_pages=self.pages, cursor=self.cursor,
            table_out=self.table, kv_lens_out=self.lens, cursor_out=self.cursor)
        gdn.gdn_page_copy([self.k, self.v], copies)
        self.status = torch.maximum(self.status, status)


def search(requests=3, beams=4, longest=90, steps=24, seed=0, end_token=1, device="cuda"):
    """Beam search; returns (scores [requests, beams], scores of the same tokens run by themselves, the stack)."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(1, longest + 1, (requests,), generator=g).tolist()
    stack = BeamStack(requests * beams, longest + steps + 1, device=device, seed=seed)
    G, K = requests, beams
    i32 = lambda v: torch.tensor(v, dtype=I32, device=device)
    prompts = [torch.randint(2, stack.vocab, (n,), generator=g) for n in lens]

    # prompts in each request's first row; the others are empty until the first selection
    prompt_lens = i32([n if k == 0 else 0 for n in lens for k in range(K)])
    logits = stack.step(torch.cat(prompts).to(device), prompt_lens, max(lens))
    ends = torch.tensor(lens).cumsum(0) - 1
    logits = logits[ends.to(device)].repeat_interleave(K, 0)
    stack.follow(i32([g * K for g in range(G) for _ in range(K)]))
    scores = torch.full((G, K), -math.inf, device=device)
    scores[:, 0] = 0
    finished = torch.zeros(G, K, dtype=torch.bool, device=device)
    ones = i32([1] * (G * K))
    history = torch.zeros(G * K, 0, dtype=I32, device=device)
    for step in range(steps):
        tokens, parents, scores, finished = gdn.gdn_beam_select(
            logits, scores, finished=finished, end_token=end_token, keep_rows=True, scores_out=scores, finished_out=finished)
        parents = parents.view(-1)
        history = torch.cat([history[parents.long()], tokens.view(-1, 1)], 1)
        stack.follow(parents)
        if step + 1 < steps:
            logits = stack.step(tokens.view(-1), ones, 1)
    status = stack.status.clone()

    # every beam's tokens again, in a row of its own from the start
    stack.reset()
    again = torch.zeros(G * K, dtype=torch.float64, device=device)
    live = torch.ones(G * K, dtype=torch.bool, device=device)
    logits = stack.step(torch.cat([p for p in prompts for _ in range(K)]).to(device), i32([n for n in lens for _ in range(K)]),
                        max(lens))
    logits = logits[(torch.tensor([n for n in lens for _ in range(K)]).cumsum(0) - 1).to(device)]
    for step in range(steps):
        token = history[:, step]
        logp = torch.log_softmax(logits.double(), -1).gather(1, token.long()[:, None])[:, 0]
        again += torch.where(live, logp, 0.0)
        live &= token != end_token
        if step + 1 < steps:
            logits = stack.step(token.contiguous(), ones, 1)
    assert status.item() == 0 and stack.status.item() == 0
    gdn.gdn_attention_status()
    return scores, again.view(G, K), history.view(G, K, steps)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--longest", type=int, default=90)
    ap.add_argument("--steps", type=int, default=24)
    a = ap.parse_args()
    scores, again, _ = search(a.requests, a.beams, a.longest, a.steps)
    for s, t in zip(scores.tolist(), again.tolist()):
        print("  ".join(f"{x:.3f} ({y:.3f})" for x, y in zip(s, t)))


if __name__ == "__main__":
    main()
