"""The device status of handles and of the 4-bit calls that take none: whose it is, and that asking
for it waits for the given stream alone."""
import threading

import pytest
import torch

from sparse_moe_layer_bias_gb300 import synth

pytestmark = pytest.mark.gpu
TIMEOUT = 6


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_moe_layer_bias_gb300 as m
    m.load_library()
    return m


def handle(lm, **cfg):
    w = {k: v.cuda() for k, v in synth.layer_weights_host(synth.TINY).items()}
    return lm.lmoe_create(dict(synth.TINY.layer_dict(), **cfg), w, max_tokens=16)


def test_a_timeout_is_reported_to_its_caller_alone(lm):
    """Waits that give up after 2 ms on a barrier that nothing arrives on, of a handle and of a call without one."""
    a, b = handle(lm, expert_w4=32), handle(lm)
    assert [lm.lmoe_device_status(a), lm.lmoe_device_status(b), lm.lmoe_w4_status()] == [0, 0, 0]
    lm.lmoe_w4_selftest_timeout(2_000_000)
    assert [lm.lmoe_device_status(a), lm.lmoe_device_status(b)] == [0, 0]
    assert [lm.lmoe_w4_status(clear=False), lm.lmoe_w4_status(), lm.lmoe_w4_status()] == [TIMEOUT, TIMEOUT, 0]
    lm.lmoe_selftest_timeout(a, 2_000_000)
    assert [lm.lmoe_w4_status(), lm.lmoe_device_status(b)] == [0, 0]
    assert [lm.lmoe_device_status(a), lm.lmoe_device_status(a)] == [TIMEOUT, 0]
    with pytest.raises(lm.LmoeError):
        lm.lmoe_w4_selftest_timeout(10)   # below 1 us: refused on the host


@pytest.mark.parametrize("ask", ["handle", "w4"])
def test_the_status_waits_for_its_stream_alone(lm, ask):
    h, side = handle(lm), torch.cuda.Stream()
    status = (lambda: lm.lmoe_device_status(h, stream=side)) if ask == "handle" else (lambda: lm.lmoe_w4_status(stream=side))
    assert status() == 0
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    torch.cuda._sleep(600_000_000)   # about a third of a second on the default stream
    done.record()
    assert status() == 0
    assert not done.query()
    torch.cuda.synchronize()


def test_the_status_leaves_another_threads_capture_alone(lm):
    h, side = handle(lm), torch.cuda.Stream()
    assert lm.lmoe_device_status(h, stream=side) == 0 and lm.lmoe_w4_status(stream=side) == 0
    t = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    got, graph = [], torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        t += 1
        other = threading.Thread(target=lambda: got.extend((lm.lmoe_device_status(h, stream=side), lm.lmoe_w4_status(stream=side))))
        other.start()
        other.join()
        t += 1
    assert got == [0, 0]
    graph.replay()
    torch.cuda.synchronize()
    assert (t == 2).all()
