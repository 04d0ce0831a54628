"""The serving example: decoding token by token over carried states and the paged cache ends
where whole sequences end.

Both ways round activations to bf16 after each of four layers and differ in the kernels they
take (token-serial and chunked recurrence, single tokens and prompts), each to within 2^-8
relative of exact arithmetic, as their own tests hold; with two roundings a layer the ends are
within 4 * 2 * 2^-8 = 3.2e-2 of each other."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    from varlen_gated_delta_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("hybrid_serving", os.path.join(ROOT, "examples", "hybrid_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("requests,longest,steps", [(1, 1, 3), (4, 300, 6), (7, 70, 5)])
def test_decoding_ends_where_whole_sequences_end(requests, longest, steps):
    out, again, _ = _example().serve(requests, longest, steps)
    assert bool(torch.isfinite(out).all())
    assert float((out.float() - again.float()).norm() / again.float().norm()) <= 3.2e-2
