"""Steps that mix single tokens with slices of prompts."""
import numpy as np
import pytest

import varlen_gated_delta_gb300 as gdn
from test_gpu_attention import BF16, _lib, check_paged, i32, make_paged  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_slice_beside_many_decode_rows_splits_its_keys():
    """63 single tokens and a slice of 64 over a long history.  Only the slice has work for the prompt kernel, whose
    items are then few: its keys are split, which shows in a launch that joins the parts."""
    news, kvs = [1] * 63 + [64], [1 + 5 * b for b in range(63)] + [4096 + 64]
    q, kc, vc, table = make_paged(news, kvs, 32, 8, 64, 64, BF16)
    args = (q, kc, vc, i32(table), i32(kvs), i32(np.concatenate([[0], np.cumsum(news)])))
    before = gdn.gdn_launch_count()
    out = gdn.gdn_attention_paged(*args, max_q=64)
    assert gdn.gdn_launch_count() - before == 4          # few rows and their join, the slice and its join
    check_paged(out, q, kc, vc, table, news, kvs, BF16)
