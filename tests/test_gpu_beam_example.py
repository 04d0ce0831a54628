"""A whole beam search: selection, states, block tables, page copies and the 4-bit cache together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_serving.py")
    spec = importlib.util.spec_from_file_location("beam_serving", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("requests,beams,longest,steps", [(1, 1, 5, 3), (3, 4, 90, 40), (5, 3, 33, 20)])
def test_beams_score_what_their_tokens_score_alone(requests, beams, longest, steps):
    scores, again, history = _example().search(requests, beams, longest, steps, seed=requests)
    # All is in fp32 but the cache.  A 4-bit code may fall to the other side of a border (some 1e-6 of 1e5 values), which
    # moves a score by about 1e-3; a state or page of another beam moves it by whole units.
    assert bool(torch.isfinite(scores).all())
    assert bool(((scores.double() - again).abs() < 0.05).all()), (scores, again)
    for beam_rows in history.tolist():
        assert len({tuple(r) for r in beam_rows}) == beams  # no two beams of a request are the same
