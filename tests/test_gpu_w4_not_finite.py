"""Weights and activations that are not finite show in the results that they reach, whichever form a
call takes, and in no other.

Quantised weights: a group that holds an infinity or a NaN has NaN weights.  In W1 or W2 that makes
one feature of the expert's activation NaN, and with it all of z for the tokens that chose the expert;
in W3 one column of z for them.  A scale that is infinite or NaN whatever its codes does the same.

Batches: 1 token runs token by token; 64 tokens of top-8 over 24 experts are grouped by expert.  A matrix
of 40000 rows takes the kernel that reads by TMA, one of 64 rows the other."""
import dataclasses

import numpy as np
import pytest
import torch

from sparse_moe_layer_bias_gb300 import synth

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_moe_layer_bias_gb300 as m
    m.load_library()
    return m


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def routing(T, E, k, seed):
    r = np.random.default_rng(seed)
    idx = np.argsort(r.normal(size=(T, E)), axis=1)[:, :k].astype(np.int32)
    return torch.from_numpy(idx), torch.from_numpy(r.uniform(0.1, 1, (T, k)).astype(np.float32))


def nan_only(got, where):
    """NaN exactly where `where` says, finite elsewhere."""
    got = got.float().cpu()
    assert torch.isnan(got[where]).all(), int((~torch.isnan(got) & where).sum())
    assert torch.isfinite(got[~where]).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", [64, 40000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m", [1, 8])
def test_matvec_with_quantised_weights_that_are_not_finite(lm, n, group, dtype, m):
    k = 1000   # (a row of scales starts anywhere)
    w = normal((n, k), 1)
    bad = {0: (3, NAN), 17: (999, INF), 33: (500, -INF), n - 1: (0, NAN)}
    for r, (c, v) in bad.items():
        w[r, c] = v
    codes, scales = lm.lmoe_w4_quantize(w.cuda(), group)
    for seed in range(4):
        y = lm.lmoe_w4_matvec(codes, scales, group, normal((m, k), seed).cuda(), out_dtype=dtype)
        where = torch.zeros(m, n, dtype=torch.bool)
        where[:, list(bad)] = True
        nan_only(y, where)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", [64, 40000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matvec_with_infinite_scales_of_any_codes(lm, n, group, dtype):
    k = 1024
    r = np.random.default_rng(n)
    codes = torch.from_numpy(r.integers(0, 256, (n, k // 2), dtype=np.uint8)).cuda()
    scales = torch.rand((n, k // group), device="cuda").to(torch.bfloat16)
    where = torch.zeros(n, dtype=torch.bool)
    for i, v in ((5, INF), (6, -INF), (7, NAN), (n - 1, INF)):
        scales[i, (i * 5) % (k // group)] = v
        where[i] = True
    for m in (1, 3, 8):
        y = lm.lmoe_w4_matvec(codes, scales, group, normal((m, k), m).cuda(), out_dtype=dtype)
        nan_only(y, where.expand(m, n))


E, K, L, I = 24, 8, 520, 136


def expert_weights(seed=5):
    return [normal((E, I, L), seed) * 0.05, normal((E, I, L), seed + 1) * 0.05, normal((E, L, I), seed + 2) * 0.05]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("T", [1, 64])
def test_experts_with_quantised_weights_that_are_not_finite(lm, T, which, value, group):
    w = expert_weights()
    idx, gates = routing(T, E, K, T)
    expert = int(idx[0, 3])
    row, col = (77, 301) if which < 2 else (301, 77)
    w[which][expert, row, col] = value
    q = [lm.lmoe_w4_quantize(t.cuda(), group) for t in w]
    for seed in range(4):   # (the residue of a group's products depends on h)
        z = lm.lmoe_w4_experts(*q, group, normal((T, L), seed).cuda(), idx.cuda(), gates.cuda())
        where = (idx == expert).any(1)[:, None].expand(T, L).clone()
        if which == 2:
            where[:, :row] = False
            where[:, row + 1:] = False
        nan_only(z, where)


@pytest.mark.parametrize("which", ["w1", "w2", "w3"])
@pytest.mark.parametrize("T", [1, 100])
def test_layer_with_weights_that_are_not_finite(lm, T, which):
    """The RMSNorm takes a NaN of z to the whole token; tokens that chose other experts stay finite."""
    shape = dataclasses.replace(synth.TINY, latent=256, inter=192)
    w = synth.layer_weights_host(shape)
    x, b = synth.activations_host(shape, T=T)
    probe = lm.lmoe_create(dict(shape.layer_dict(), expert_w4=32), {k: v.cuda() for k, v in w.items()}, max_tokens=T)
    idx = torch.empty((T, shape.top_k), dtype=torch.int32, device="cuda")
    lm.lmoe_forward(probe, x.cuda(), b.cuda(), topk_idx_out=idx)
    expert = int(idx[0, 0])
    w[which] = w[which].clone()
    w[which][expert, 100, 31] = INF
    h = lm.lmoe_create(dict(shape.layer_dict(), expert_w4=32), {k: v.cuda() for k, v in w.items()}, max_tokens=T)
    y = lm.lmoe_forward(h, x.cuda(), b.cuda())
    nan_only(y, (idx.cpu() == expert).any(1)[:, None].expand(T, shape.d))
    for one in (probe, h):
        lm.lmoe_destroy(one)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("n", [64, 40000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k", [1000, 1001])
@pytest.mark.parametrize("m", [1, 3, 8, 20])
def test_matvec_with_activations_that_are_not_finite(lm, n, k, group, dtype, m):
    """A row of x with an infinity gives NaN throughout its row of y, as one with a NaN does, in every form."""
    codes, scales = lm.lmoe_w4_quantize(normal((n, k), 1).cuda(), group)
    for at, value in ((0, INF), (k // 2, -INF), (k - 1, NAN)):
        x = normal((m, k), at)
        row = at % m
        x[row, at] = value
        where = torch.zeros(m, n, dtype=torch.bool)
        where[row] = True
        nan_only(lm.lmoe_w4_matvec(codes, scales, group, x.cuda(), out_dtype=dtype), where)


@pytest.mark.parametrize("T", [1, 64])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_experts_with_activations_that_are_not_finite(lm, T, value):
    q = [lm.lmoe_w4_quantize(t.cuda(), 32) for t in expert_weights()]
    idx, gates = routing(T, E, K, T)
    h = normal((T, L), 3)
    t = T // 2
    h[t, 111] = value
    where = torch.zeros(T, L, dtype=torch.bool)
    where[t] = True
    nan_only(lm.lmoe_w4_experts(*q, 32, h.cuda(), idx.cuda(), gates.cuda()), where)
