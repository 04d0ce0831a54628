"""Packed prompts of thousands of tokens against the definition in 64 bits, and calls with room for so many tokens that
the items' order has several places of a sequence to a bin.  Tolerances as in test_gpu_attention."""
import math

import numpy as np
import pytest
import torch

import varlen_gated_delta_gb300 as gdn
from test_gpu_attention import BF16, DEV, F32, _lib, check, gen, i32, rand, run_varlen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("H,HKV,D", [(4, 2, 128), (3, 3, 64), (2, 1, 256)])
def test_long_prompts(dt, H, HKV, D):
    lens = [5000, 1, 2049, 900, 3328]
    offs = np.concatenate([[0], np.cumsum(lens)])
    g = gen(D)
    q, k, v = rand(g, int(offs[-1]), H, D, dt=dt, std=2.0), *(rand(g, int(offs[-1]), HKV, D, dt=dt) for _ in "kv")
    out = gdn.gdn_attention_varlen(q, k, v, i32(offs))
    for b, n in enumerate(lens):
        rows = slice(int(offs[b]), int(offs[b + 1]))
        want, mag = (torch.empty(n, H, D, dtype=torch.float64) for _ in range(2))
        hidden = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)
        for h in range(H):
            x = (q[rows, h].double() @ k[rows, h // (H // HKV)].double().T) / math.sqrt(D)
            p = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            vals = v[rows, h // (H // HKV)].double()
            want[:, h], mag[:, h] = (p @ vals).cpu(), (p @ vals.abs()).cpu()
        check(out[rows], want, mag, dt, f"sequence {b}")


@pytest.mark.parametrize("room", [530_000, 1_100_000])
def test_room_for_many_more_tokens_than_there_are(room):
    """Query tiles of 128 tokens: two (four) neighbouring ones of a sequence share a bin of the order."""
    run_varlen([700, 1, 300, 0, 129, 1500], 2, 1, 64, BF16, seed=room, extra_rows=room)
