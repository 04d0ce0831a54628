"""The binding of the softmax-attention calls, without a GPU."""
import contextlib

import pytest
import torch

import varlen_gated_delta_gb300 as gdn
from varlen_gated_delta_gb300 import build as gdn_build


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


@pytest.fixture
def unbuildable(monkeypatch, tmp_path):
    """A machine on which the compiled part of the binding does not build: a header is missing."""
    source = tmp_path / "marshal.cpp"
    source.write_text("#include <no_such_header_of_python.h>\n")
    monkeypatch.setattr(gdn_build, "MARSHAL_SRC", str(source))
    monkeypatch.setattr(gdn_build, "marshal_path", lambda: str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(gdn, "_marshal_module", None)


def test_the_library_is_built_without_the_compiled_part_of_the_binding(unbuildable):
    """The delta calls need neither Python's nor torch's headers."""
    with pytest.warns(RuntimeWarning, match="no_such_header_of_python"):
        assert gdn_build.build() == gdn_build.LIB
    assert gdn.load_library().gdn_version() > 0
    with pytest.raises(gdn.GdnError, match="is missing") as e:
        gdn.gdn_attention_varlen(*[torch.zeros(1)] * 4)
    assert e.value.status == 6


def test_the_library_is_built_without_a_host_compiler_for_the_binding(unbuildable, monkeypatch, tmp_path):
    monkeypatch.setattr(gdn_build.shutil, "which", lambda name: str(tmp_path / name))
    monkeypatch.setattr(gdn_build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    with pytest.warns(RuntimeWarning):
        assert gdn_build.build() == gdn_build.LIB
