"""The compiled calls as a Python program meets them: gradients they cannot give, other threads, memory that
is not there."""
import threading
import time

import pytest
import torch

import gated_deltanet_gdn_gb300 as gdn

from paged_reference import Paged

pytestmark = pytest.mark.gpu


def _setup():
    c = Paged([3, 1], [20, 40], 4, 2, 64, 16, "bf16", seed=41)
    q, k, v = (c.normal(4, h, 64).cuda() for h in (4, 2, 2))
    return q, k, v, c.cuda()


@pytest.mark.parametrize("name", ["q", "k_cache", "v_cache", "out"])
def test_attention_refuses_to_lose_a_gradient(name):
    q, _, _, (kc, vc, *where) = _setup()
    t = dict(q=q, k_cache=kc, v_cache=vc, out=torch.empty_like(q))

    def call():
        return gdn.gdn_paged_attn(t["q"], t["k_cache"], t["v_cache"], *where, 0.1, max_q=3, max_kv=40, out=t["out"])

    plain = call().clone()
    t[name].requires_grad_()
    with pytest.raises(gdn.GdnError, match=name):
        call()
    with torch.no_grad():
        assert torch.equal(call(), plain)
    with torch.inference_mode():
        assert torch.equal(call(), plain)
    t[name] = t[name].detach()
    assert torch.equal(call(), plain)


@pytest.mark.parametrize("name", ["q", "k", "v", "k_cache", "v_cache", "q_out"])
def test_append_refuses_to_lose_a_gradient(name):
    q, k, v, (kc, vc, *where) = _setup()
    t = dict(q=q, k=k, v=v, k_cache=kc, v_cache=vc, q_out=torch.empty_like(q))

    def call():
        return gdn.gdn_kv_append(t["k"], t["v"], t["k_cache"], t["v_cache"], *where, q=t["q"], q_out=t["q_out"])

    plain = call().clone()
    t[name].requires_grad_()
    with pytest.raises(gdn.GdnError, match=name):
        call()
    with torch.no_grad():
        assert torch.equal(call(), plain)


def test_other_threads_run_while_a_launch_waits():
    """More launches than the queue holds behind a kernel of about a second: the launching thread waits, and a
    second thread keeps its turns."""
    _, k, v, (kc, vc, *where) = _setup()
    gdn.gdn_kv_append(k, v, kc, vc, *where)
    torch.cuda.synchronize()
    stop, gap = threading.Event(), [0.0]

    def watch():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gap[0] = max(gap[0], now - last)
            last = now

    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    torch.cuda._sleep(1_800_000_000)
    end.record()
    t = threading.Thread(target=watch)
    t.start()
    try:
        for _ in range(6000):
            gdn.gdn_kv_append(k, v, kc, vc, *where)
    finally:
        stop.set()
        t.join()
        torch.cuda.synchronize()
    span = start.elapsed_time(end) / 1e3
    assert span > 0.5  # the queue was full for most of this
    assert gap[0] < span / 4, (gap[0], span)


def test_out_of_memory_is_pytorchs_error():
    """Outputs beyond the process's share of the memory: the error that programs catch to try a smaller batch."""
    x = torch.zeros(1, 1, 4096, device="cuda").expand(1 << 20, 1, 4096)  # 16 GB as a contiguous output
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 30)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            gdn.gdn_block_norm_fwd(x)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
