"""Serving a small stack of gated-delta and softmax-attention layers.

Every other layer is a gated-delta layer (conv and recurrent state per request), the
others are causal attention over a paged key-value cache.  A batch of ragged prompts
is taken in packed, then tokens are decoded one at a time for all requests:

  per step       gdn_page_plan: pages, slots and positions of the new tokens, with the
                 lengths and the page cursor carried in place on the device
  delta layer    gdn_layer_varlen, conv and delta states carried in place
  attention      gdn_qk_norm_rope writes k and v to the cache; gdn_attention_varlen for
                 prompts, gdn_attention_paged for single tokens

Weights are random.  At the end the prompts and the decoded inputs are run again as
whole sequences, and the last hidden states of both ways are compared.

  python examples/hybrid_serving.py [--requests 4] [--longest 300] [--steps 16]
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import varlen_gated_delta_gb300 as gdn  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class HybridStack:
    """`layers` layers, even ones gated delta, odd ones attention, for up to `requests` requests."""

    def __init__(self, requests, max_tokens, layers=4, width=512, HQ=2, H=4, AH=8, AHKV=2, D=128, page_size=64,
                 device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.rand = lambda *s, std=1.0, dt=BF16: (torch.randn(*s, generator=g, device=device) * std).to(dt)
        self.dev, self.B, self.width, self.ps = device, requests, width, page_size
        self.HQ, self.H, self.AH, self.AHKV, self.D = HQ, H, AH, AHKV, D
        W = 2 * HQ * D + H * D                     # the delta layer's packed q, k, v channels
        lin = lambda i, o: self.rand(i, o, std=1 / math.sqrt(i))
        self.layers = []
        for n in range(layers):
            if n % 2 == 0:
                self.layers.append(dict(
                    kind="delta", qkv=lin(width, W), gates=lin(width, 2 * H), out=lin(H * D, width),
                    conv=self.rand(W, 4, std=0.5), A_log=torch.rand(H, generator=g, device=device) * math.log(16.0),
                    dt_bias=self.rand(H, dt=F32)))
            else:
                self.layers.append(dict(
                    kind="attention", qkv=lin(width, (AH + 2 * AHKV) * D), out=lin(AH * D, width),
                    qw=1 + 0.1 * self.rand(D, dt=F32), kw=1 + 0.1 * self.rand(D, dt=F32)))
        angle = (torch.arange(max_tokens, dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)[None, :])
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)
        self.max_pages = -(-max_tokens // page_size)
        self.reset()

    def reset(self):
        """Empty states, caches and page tables."""
        self.empty = True
        B, D, dev = self.B, self.D, self.dev
        pages = B * self.max_pages
        for L in self.layers:
            if L["kind"] == "delta":
                L["conv_state"] = torch.zeros(B, L["conv"].shape[0], 3, device=dev, dtype=BF16)
                L["state"] = torch.zeros(B, self.H, D, D, device=dev)
            else:
                L["k"], L["v"] = (torch.zeros(pages, self.ps, self.AHKV, D, device=dev, dtype=BF16) for _ in "kv")
        self.lens = torch.zeros(B, dtype=I32, device=dev)
        self.table = torch.full((B, self.max_pages), -1, dtype=I32, device=dev)
        self.free = torch.arange(pages, dtype=I32, device=dev)
        self.cursor = torch.zeros(1, dtype=I32, device=dev)

    def step(self, x, new_lens, longest):
        """Hidden states [N, width] of new_lens[b] new tokens of each request, through all layers.
        `longest` is the largest of new_lens; a first step takes whole prompts."""
        N, H, HQ, D = x.shape[0], self.H, self.HQ, self.D
        first, self.empty = self.empty, False
        offsets, _, positions, slots, _, status = gdn.gdn_page_plan(
            new_lens, self.lens, self.table, self.free, page_size=self.ps, N=N, cursor=self.cursor, kv_lens=self.lens,
            cursor_out=self.cursor)
        for L in self.layers:
            h = torch.nn.functional.rms_norm(x, (self.width,))
            if L["kind"] == "delta":
                a, b = (h @ L["gates"]).float().split(H, 1)
                y, _, _ = gdn.gdn_layer_varlen(
                    h @ L["qkv"], L["conv"], None, a.contiguous(), b.contiguous(), L["A_log"], L["dt_bias"], offsets,
                    L["conv_state"], L["state"], H=H, HQ=HQ, K=D, V=D, conv_fin=L["conv_state"], state_fin=L["state"])
            else:
                qkv = h @ L["qkv"]
                k = torch.empty(N, self.AHKV, D, device=self.dev, dtype=BF16) if first else None
                q, k = gdn.gdn_qk_norm_rope(qkv, self.cos_sin, positions, H=self.AH, HKV=self.AHKV, D=D,
                                            q_weight=L["qw"], k_weight=L["kw"], k=k, slots=slots, k_cache=L["k"],
                                            v_cache=L["v"])
                if first:   # nothing cached before: the prompts' own keys and values, v in place in the projection
                    v = qkv[:, (self.AH + self.AHKV) * D:].view(N, self.AHKV, D)
                    y = gdn.gdn_attention_varlen(q, k, v, offsets)
                else:
                    y = gdn.gdn_attention_paged(q, L["k"], L["v"], self.table, self.lens, offsets, max_q=longest)
            x = x + y.reshape(N, -1) @ L["out"]
        self.status = status
        return x


def serve(requests=4, longest=300, steps=16, seed=0, device="cuda"):
    """Prompts, then `steps` decode steps; returns (last hidden states, the same from whole sequences, seconds)."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(1, longest + 1, (requests,), generator=g).tolist()
    stack = HybridStack(requests, longest + steps + 1, device=device, seed=seed)
    prompts = [stack.rand(n, stack.width) for n in lens]
    tokens = [stack.rand(requests, stack.width) for _ in range(steps)]
    i32 = lambda v: torch.tensor(v, dtype=I32, device=device)

    stack.step(torch.cat(prompts), i32(lens), max(lens))
    ones = i32([1] * requests)
    torch.cuda.synchronize()
    began = time.perf_counter()
    for x in tokens:
        out = stack.step(x, ones, 1)
    torch.cuda.synchronize()
    seconds = time.perf_counter() - began
    assert stack.status.item() == 0 and stack.lens.tolist() == [n + steps for n in lens]

    stack.reset()
    whole = [torch.cat([p] + [t[b:b + 1] for t in tokens]) for b, p in enumerate(prompts)]
    again = stack.step(torch.cat(whole), i32([len(w) for w in whole]), max(len(w) for w in whole))
    ends = torch.tensor([len(w) for w in whole]).cumsum(0) - 1
    gdn.gdn_attention_status()
    return out, again[ends.to(device)], seconds


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--longest", type=int, default=300)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    out, again, seconds = serve(a.requests, a.longest, a.steps)
    far = float((out.float() - again.float()).norm() / again.float().norm())
    print(f"{a.requests} requests, {a.steps} steps: {seconds / a.steps * 1e6:.0f} us a step; "
          f"decoded against whole sequences: {far:.1e} apart")


if __name__ == "__main__":
    main()
