"""Calls from host threads other than the one that set up the GPU."""
import ctypes
import dataclasses
import threading

import pytest
import torch

from sparse_moe_layer_bias_gb300 import binding, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_moe_layer_bias_gb300 as m
    m.load_library()
    return m


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def w4(lm, n, k, lead=()):
    codes, scales = lm.lmoe_w4_quantize(torch.randn(*lead, n, k, device="cuda").to(torch.bfloat16), 32)
    return binding.LmoeW4(codes.data_ptr(), scales.data_ptr(), codes.shape[-1], scales.shape[-1]), (codes, scales)


def matvec(lm, n, k):
    """A call of lmoe_w4_matvec on a stream as a function that gives its status, its output and what that should be."""
    lib, (w, kept) = lm.load_library(), w4(lm, n, k)
    x, y = torch.randn(8, k, device="cuda").to(torch.bfloat16), torch.empty(8, n, dtype=torch.bfloat16, device="cuda")
    call = lambda s: lib.lmoe_w4_matvec(ctypes.byref(w), n, k, 32, ptr(x), 8, k, ptr(y), n, 0, s)
    return call, y, lm.lmoe_w4_matvec(*kept, 32, x), (w, kept, x)


def experts(lm, T, L, I):
    lib, stacks = lm.load_library(), [w4(lm, n, k, (16,)) for n, k in ((I, L), (I, L), (L, I))]
    h = torch.randn(T, L, device="cuda").to(torch.bfloat16)
    idx = torch.rand(T, 16, device="cuda").argsort(1)[:, :8].int().contiguous()
    gates, z = torch.rand(T, 8, device="cuda"), torch.empty_like(h)
    ws = torch.empty(lm.lmoe_w4_experts_workspace_size(T, 8, 16, L, I), dtype=torch.uint8, device="cuda")
    call = lambda s: lib.lmoe_w4_experts(*[ctypes.byref(w) for w, _ in stacks], 16, L, I, 32, ptr(h), T, ptr(idx), ptr(gates), 8,
                                         4.0, 25.0, ptr(z), ptr(ws), ws.numel(), s)
    return call, z, lm.lmoe_w4_experts(*[q for _, q in stacks], 32, h, idx, gates), (stacks, h, idx, gates, ws)


def layer(lm, T, shape=synth.TINY, **cfg):
    lib = lm.load_library()
    w = {k: v.cuda() for k, v in synth.layer_weights_host(shape).items()}
    x, b = (t.cuda() for t in synth.activations_host(shape, T=T))
    h = lm.lmoe_create(dict(shape.layer_dict(), **cfg), w, max_tokens=T)
    ws, y = lm.alloc_workspace(h, T), torch.empty_like(x)
    call = lambda s: lib.lmoe_forward(h.ptr, ptr(x), T, ptr(b), ptr(y), None, None, None, None, ptr(ws), ws.numel(), s)
    return call, y, lm.lmoe_forward(h, x, b), (h, w, x, b, ws)


def in_thread(f):
    got = []
    t = threading.Thread(target=lambda: got.append(f()))
    t.start()
    t.join()
    return got[0]


@pytest.mark.parametrize("make", [lambda lm: matvec(lm, 40000, 512), lambda lm: experts(lm, 64, 256, 96), lambda lm: layer(lm, 48),
                                  lambda lm: layer(lm, 48, expert_w4=32)], ids=["matvec", "experts", "layer", "layer_w4"])
def test_the_first_call_of_a_thread(lm, make):
    """A thread in which no other CUDA call has been made."""
    call, y, want, _ = make(lm)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    y.zero_()
    torch.cuda.synchronize()
    assert in_thread(lambda: call(ctypes.c_void_p(stream.cuda_stream))) == 0
    stream.synchronize()
    assert torch.equal(y, want)


def test_a_backward_as_the_first_call_of_a_thread(lm):
    shape, T = synth.TINY, 48
    w = {k: v.cuda() for k, v in synth.layer_weights_host(shape).items()}
    x, b = (t.cuda() for t in synth.activations_host(shape, T=T))
    dy = synth.grad_output_host(shape, T=T).cuda()
    h = lm.lmoe_create(dict(shape.layer_dict(), with_backward=True), w, max_tokens=T)
    ws = lm.alloc_workspace(h, T)
    lm.lmoe_forward(h, x, b, workspace=ws)
    dx, want = torch.empty_like(x), lm.lmoe_backward(h, x, dy, ws)[0]
    grads = {n: torch.empty(s, device="cuda") for n, s in lm.grad_shapes(h).items()}
    g = binding.LmoeGrads(*[grads[n].data_ptr() for n in binding.WEIGHT_NAMES], 0)
    bws = torch.empty(lm.lmoe_backward_workspace_size(h, T), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    lib = lm.load_library()
    assert in_thread(lambda: lib.lmoe_backward(h.ptr, ptr(x), T, ptr(dy), None, None, ptr(ws), ws.numel(), ptr(dx), ctypes.byref(g),
                                               ptr(bws), bws.numel(), None)) == 0
    torch.cuda.synchronize()
    assert torch.equal(dx, want)


def run_threads(calls, repeats):
    """Each of `calls` `repeats` times in a thread and on a stream of its own; the statuses that are not 0."""
    start, bad = threading.Barrier(len(calls)), []
    streams = [torch.cuda.Stream() for _ in calls]

    def loop(call, stream):
        start.wait()
        for _ in range(repeats):
            st = call(ctypes.c_void_p(stream.cuda_stream))
            if st:
                bad.append(st)

    threads = [threading.Thread(target=loop, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


def check_together(made, repeats):
    """Calls of different sizes at once: none disturbs another's launch (what a launch sets on a kernel, such as its
    limit of shared memory, is seen by all threads; ctypes lets go of the interpreter during a call, so they do overlap)."""
    torch.cuda.synchronize()
    assert not run_threads([m[0] for m in made], repeats)
    for _, y, want, _ in made:
        assert torch.equal(y, want)


@pytest.mark.parametrize("n", [64, 30000])
def test_matvecs_of_different_widths_at_once(lm, n):
    check_together([matvec(lm, n, k) for k in (64, 700, 2048, 5000)], 3000)


def test_experts_of_different_widths_at_once(lm):
    check_together([experts(lm, *a) for a in ((64, 64, 32), (64, 2048, 64), (64, 512, 1500), (1, 3584, 512), (2, 64, 40))], 1000)


def test_layers_of_different_widths_at_once(lm):
    """top_k and latent set the sizes of the sum over a token's experts."""
    tiny = synth.TINY
    made = [layer(lm, 8, dataclasses.replace(tiny, latent=latent, top_k=k)) for latent, k in ((128, 1), (512, 4), (1024, 16), (2048, 30))]
    made += [layer(lm, 8, dataclasses.replace(tiny, latent=latent), expert_w4=32) for latent in (256, 1536)]
    check_together(made, 300)


def backward(lm, shape, T):
    lib = lm.load_library()
    w = {k: v.cuda() for k, v in synth.layer_weights_host(shape).items()}
    x, b = (t.cuda() for t in synth.activations_host(shape, T=T))
    dy = synth.grad_output_host(shape, T=T).cuda()
    h = lm.lmoe_create(dict(shape.layer_dict(), with_backward=True), w, max_tokens=T)
    ws, dx = lm.alloc_workspace(h, T), torch.empty_like(x)
    lm.lmoe_forward(h, x, b, workspace=ws)
    want = lm.lmoe_backward(h, x, dy, ws)[0]
    grads = {n: torch.empty(s, device="cuda") for n, s in lm.grad_shapes(h).items()}
    g = binding.LmoeGrads(*[grads[n].data_ptr() for n in binding.WEIGHT_NAMES], 0)
    bws = torch.empty(lm.lmoe_backward_workspace_size(h, T), dtype=torch.uint8, device="cuda")
    call = lambda s: lib.lmoe_backward(h.ptr, ptr(x), T, ptr(dy), None, None, ptr(ws), ws.numel(), ptr(dx), ctypes.byref(g),
                                       ptr(bws), bws.numel(), s)
    return call, dx, want, (h, w, x, b, dy, ws, grads, bws)


def test_backwards_of_different_widths_at_once(lm):
    check_together([backward(lm, dataclasses.replace(synth.TINY, latent=latent), 8) for latent in (128, 512, 2048)], 100)


def test_histograms_of_different_bins_at_once(lm):
    lib, made = lm.load_library(), []
    for E, B in ((64, 100), (64, 1000), (64, 3000), (61, 50), (61, 4000)):
        s = torch.rand(300, E, device="cuda")
        hist = torch.empty((E, B), dtype=torch.int32, device="cuda")
        made.append((lambda st, s=s, E=E, B=B, hist=hist: lib.qb_histogram(ptr(s), 300, E, E, B, ptr(hist), 0, st), hist,
                     lm.qb_histogram(s, B), s))
    check_together(made, 2000)
