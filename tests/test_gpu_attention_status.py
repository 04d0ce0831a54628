"""A wait of the attention kernels that runs out, without a GPU fault: it is reported to every stream that asks, once,
and later calls are whole."""
import pytest
import torch

import varlen_gated_delta_gb300 as gdn
from test_gpu_attention import BF16, _lib, run_paged, run_varlen  # noqa: F401

pytestmark = pytest.mark.gpu


def timed_out():
    try:
        gdn.gdn_attention_status()
    except gdn.GdnError as e:
        assert e.status == 7
        return True
    return False


def test_a_wait_that_gives_up_is_reported_once():
    timed_out()
    gdn.gdn_selftest_attention_timeout(2000)
    assert timed_out() and not timed_out()
    run_varlen([130, 40], 4, 2, 128, BF16)
    run_paged([1, 70], [300, 400], 4, 2, 128, 16, BF16)
    assert not timed_out()


def test_no_query_takes_a_report_from_another_stream():
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (side, other):
        with torch.cuda.stream(s):
            timed_out()
    timed_out()
    with torch.cuda.stream(side):
        gdn.gdn_selftest_attention_timeout(1000)
    side.synchronize()
    seen = [timed_out()]
    for s in (other, side):
        with torch.cuda.stream(s):
            seen += [timed_out(), timed_out()]
    assert seen == [True, True, False, True, False]
    assert not timed_out()


@pytest.mark.parametrize("limit_us", [5000, 100000])
def test_a_wait_lasts_about_as_long_as_its_tries(limit_us):
    """A wait counts its tries, not the clock.  A try takes up to 3.8 us and is taken for 4."""
    gdn.gdn_selftest_attention_timeout(10)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    gdn.gdn_selftest_attention_timeout(limit_us)
    b.record()
    assert timed_out()
    assert 0.25 * limit_us <= a.elapsed_time(b) * 1e3 <= 2 * limit_us + 50000


@pytest.mark.parametrize("limit", [0, -1, 1000001])
def test_refusals(limit):
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_selftest_attention_timeout(limit)
    assert e.value.status == 2
