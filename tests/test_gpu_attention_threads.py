"""The attention-layer calls beside other Python threads."""
import threading
import time

import pytest
import torch

import varlen_gated_delta_gb300 as gdn
from test_gpu_attention import BF16, DEV, _lib, gen, i32, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def calls():
    g = gen(0)
    H, HKV, D, ps, B = 4, 2, 64, 16, 3
    q, k, v, kc, vc = (rand(g, *s) for s in ((B, H, D), (B, HKV, D), (B, HKV, D), (8, ps, HKV, D), (8, ps, HKV, D)))
    qkv, out, qo = rand(g, B, (H + 2 * HKV) * D), torch.empty(B, H, D, device=DEV, dtype=BF16), rand(g, B, H, D)
    offs, ones, lens, cursor = i32([0, 1, 2, 3]), i32([1] * B), i32([4] * B), i32([0])
    table, free = i32([[0, 1], [2, 3], [4, 5]]), i32(range(8))
    plan = dict(offsets=i32([0] * 4), kv_lens=i32([0] * 3), positions=i32([0] * 3), slots=i32([0] * 3), cursor_out=i32([0]),
                status=i32([0]))
    ws = torch.empty(gdn.gdn_attention_paged_workspace_bytes(B, B, H, HKV, D, 1), dtype=torch.uint8, device=DEV)
    return dict(
        plan=lambda: gdn.gdn_page_plan(ones, lens, table, free, page_size=ps, N=B, cursor=cursor, **plan),
        rope=lambda: gdn.gdn_qk_norm_rope(qkv, H=H, HKV=HKV, D=D, q=qo, slots=offs[:3],
                                          k_cache=kc, v_cache=vc),
        varlen=lambda: gdn.gdn_attention_varlen(q, k, v, offs, out=out),
        paged=lambda: gdn.gdn_attention_paged(q, kc, vc, table, lens, offs, max_q=1, out=out, workspace=ws))


@pytest.mark.parametrize("name", ["plan", "rope", "varlen", "paged"])
def test_other_threads_run_while_a_call_waits_for_room_in_the_launch_queue(name):
    """The device is kept busy for some 0.3 s and calls are made until one of them has to wait for it: meanwhile
    another Python thread goes on."""
    call = calls()[name]
    call()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)

    thread = threading.Thread(target=tick)
    thread.start()
    longest = (0.0, 0.0, 0.0)
    torch.cuda._sleep(600_000_000)
    for _ in range(6000):
        t0 = time.perf_counter()
        call()
        t1 = time.perf_counter()
        longest = max(longest, (t1 - t0, t0, t1))
        if longest[0] > 0.05:
            break
    stop.set()
    thread.join()
    torch.cuda.synchronize()
    if longest[0] <= 0.05:
        pytest.skip("no call had to wait")
    during = sum(longest[1] < t < longest[2] for t in ticks)
    assert during >= 5, f"{during} ticks during a call of {longest[0]:.3f} s"
