"""The binding of the softmax-attention calls, without a GPU."""
import contextlib

import pytest
import torch

import varlen_gated_delta_gb300 as gdn


@pytest.mark.parametrize("device", [1, "cuda:1", torch.device("cuda", 1)], ids=str)
def test_attention_status_asks_the_device_that_it_is_given(monkeypatch, device):
    """The C call asks the current device, through a stream that must be its own."""
    current, asked = [0], []

    @contextlib.contextmanager
    def made_current(d):
        before, current[0] = current[0], torch.device(d).index if not isinstance(d, int) else d
        yield
        current[0] = before

    class Library:
        def gdn_attention_status(self, stream):
            asked.append((current[0], stream))
            return 0

    monkeypatch.setattr(torch.cuda, "device", made_current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(gdn, "_stream", lambda d: 100 + (torch.device(d).index if not isinstance(d, int) else d))
    monkeypatch.setattr(gdn, "load_library", Library)
    gdn.gdn_attention_status(device)
    gdn.gdn_attention_status()
    assert asked == [(1, 101), (0, 100)] and current == [0]
