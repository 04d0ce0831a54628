"""A malformed sequence beside sound ones, where the keys of a call are split over CTAs and joined: only
the malformed one is skipped.  Tolerances as in test_gpu_attention."""
import pytest
import torch

import varlen_gated_delta_gb300 as gdn
from test_gpu_attention import BF16, DEV, F32, SENTINEL, _lib, check_paged, i32, make_paged  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,n", [(F32, 1), (F32, 5), (F32, 70), (BF16, 1), (BF16, 5), (BF16, 70)])
@pytest.mark.parametrize("ends,sound", [
    (lambda n: [0, n, 3 * n + 50], [0]),                        # the last sequence ends past N
    (lambda n: [0, n, 3 * n + 60, n, 2 * n], [0, 3]),           # in the middle one past N, then one of negative length
    (lambda n: [0, n, 2 * n, n - 1], [0, 1]),                   # the last entry is too small
    (lambda n: [-1, n, 2 * n], [1]),                            # the first entry is not in range
], ids=["past-N", "middle", "last-too-small", "negative"])
def test_split_keys_beside_a_malformed_sequence(dt, n, ends, sound):
    offs = ends(n)
    kvs = [900 + n, 700 + n, 40 + n, 600 + n][:len(offs) - 1]
    # a table of 3200 keys, so that fp32 and the slices split them
    q, kc, vc, table = make_paged([n] * len(kvs), kvs, 4, 2, 64, 16, dt, max_pages=200)
    q = q[:3 * n].contiguous()
    out = torch.full(q.shape, SENTINEL, device=DEV, dtype=dt)
    gdn.gdn_attention_paged(q, kc, vc, i32(table), i32(kvs), i32(offs), max_q=n, out=out)
    written = torch.zeros(q.shape[0], dtype=torch.bool, device=DEV)
    for b in sound:
        rows = slice(offs[b], offs[b + 1])
        check_paged(out[rows], q[rows], kc, vc, table[b:b + 1], [n], [kvs[b]], dt, what=str(b))
        written[rows] = True
    assert bool((out[~written] == SENTINEL).all())
