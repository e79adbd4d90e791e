"""The balance loss and the 4-bit products refuse bad arguments before any CUDA
call (so this runs without a GPU), and the binding refuses tensors that do not
fit."""
import ctypes

import pytest
import torch

from sparse_moe_layer_bias_gb300 import binding, build

INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
A = 4096   # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def balance(lib, **kw):
    a = dict(scores=A, T=8, E=16, ld=16, idx=A, k=2, off=None, G=1, mask=None, norm=1, coef=1.0, dloss=None, loss=A,
             counts=None, dscores=None, ldd=0, acc=0, ws=A, wsb=1 << 30)
    a.update(kw)
    return lib.lmoe_balance_loss(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(ld=15), INVALID), (dict(loss=None), INVALID),
    (dict(ws=None), INVALID), (dict(scores=None), INVALID), (dict(idx=None), INVALID), (dict(G=0, off=A), INVALID),
    (dict(G=2), INVALID), (dict(norm=2), INVALID), (dict(acc=2), INVALID), (dict(coef=float("nan")), INVALID),
    (dict(dscores=A, ldd=15), INVALID), (dict(E=1025, ld=1025), SHAPE), (dict(k=33, E=64, ld=64), SHAPE),
    (dict(k=17), SHAPE), (dict(T=1 << 31), SHAPE), (dict(scores=A + 4), ALIGN), (dict(mask=A + 1), ALIGN),
    (dict(ws=A + 16), ALIGN), (dict(dscores=A + 8, ldd=16), ALIGN), (dict(wsb=100), WORKSPACE)])
def test_balance_loss_refuses(lib, change, status):
    assert balance(lib, **change) == status


def test_balance_workspace_size(lib):
    n = ctypes.c_size_t()
    assert lib.lmoe_balance_loss_workspace_size(896, 0, ctypes.byref(n)) == INVALID
    assert lib.lmoe_balance_loss_workspace_size(1025, 1, ctypes.byref(n)) == SHAPE
    assert lib.lmoe_balance_loss_workspace_size(896, 1, None) == INVALID
    sizes = []
    for g in (1, 2, 100):
        assert lib.lmoe_balance_loss_workspace_size(896, g, ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[0] >= 4 * 896
    assert balance(lib, E=896, ld=896, G=100, off=A, wsb=sizes[2] - 1) == WORKSPACE


def w4(codes=A, scales=A, ld_codes=64, ld_scales=4):
    return binding.LmoeW4(codes, scales, ld_codes, ld_scales)


def matvec(lib, w=None, **kw):
    a = dict(n=16, k=128, group=32, x=A, m=1, ldx=128, y=A, ldy=16, f32=0)
    a.update(kw)
    w = w4() if w is None else w
    return lib.lmoe_w4_matvec(ctypes.byref(w), *a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(m=-1), INVALID), (dict(group=48), INVALID), (dict(ldx=127), INVALID),
    (dict(ldy=15), INVALID), (dict(f32=2), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(m=65), SHAPE), (dict(k=65537, ldx=65537), SHAPE), (dict(x=A + 2), ALIGN), (dict(y=A + 2), ALIGN),
    (dict(w=w4(codes=None)), INVALID), (dict(w=w4(ld_codes=60)), INVALID), (dict(w=w4(ld_codes=48)), INVALID),
    (dict(w=w4(ld_scales=3)), INVALID), (dict(w=w4(codes=A + 8)), ALIGN), (dict(w=w4(scales=A + 2)), ALIGN)])
def test_w4_matvec_refuses(lib, change, status):
    assert matvec(lib, **change) == status


def test_w4_matvec_without_tokens_does_nothing(lib):
    assert matvec(lib, m=0, x=None, y=None) == 0


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(k=0), INVALID), (dict(ldw=127), INVALID), (dict(group=16), INVALID),
    (dict(w=None), INVALID), (dict(codes=None), INVALID), (dict(ldc=80, k=200, ldw=200), INVALID), (dict(lds=3), INVALID),
    (dict(k=65537, ldw=65537), SHAPE), (dict(w=A + 2), ALIGN), (dict(codes=A + 4), ALIGN)])
def test_w4_quantize_refuses(lib, change, status):
    a = dict(w=A, rows=16, k=128, ldw=128, group=32, codes=A, ldc=64, scales=A, lds=4)
    a.update(change)
    assert lib.lmoe_w4_quantize(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(T=-1), INVALID), (dict(beta1=0.0), INVALID),
    (dict(beta2=float("nan")), INVALID), (dict(group=31), INVALID), (dict(h=None), INVALID), (dict(z=None), INVALID),
    (dict(idx=None), INVALID), (dict(gates=None), INVALID), (dict(ws=None), INVALID), (dict(w2=w4(ld_codes=80)), INVALID),
    (dict(w2=w4(ld_scales=5)), INVALID), (dict(w3=w4(ld_scales=1)), INVALID), (dict(T=1025), SHAPE), (dict(k=33), SHAPE),
    (dict(E=1025), SHAPE), (dict(L=32769), SHAPE), (dict(h=A + 2), ALIGN), (dict(ws=A + 16), ALIGN),
    (dict(wsb=100), WORKSPACE)])
def test_w4_experts_refuses(lib, change, status):
    a = dict(w1=w4(), w2=w4(), w3=w4(), E=8, L=128, I=64, group=32, h=A, T=4, idx=A, gates=A, k=2, beta1=4.0, beta2=25.0,
             z=A, ws=A, wsb=1 << 30)
    a.update(change)
    for n in ("w1", "w2", "w3"):
        a[n] = ctypes.byref(a[n])
    assert lib.lmoe_w4_experts(*a.values(), None) == status


def test_w4_experts_workspace_never_shrinks(lib):
    n, sizes = ctypes.c_size_t(), []
    for T in (0, 1, 2, 3, 64, 1024):
        assert lib.lmoe_w4_experts_workspace_size(T, 16, 896, 3584, 512, ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert sizes == sorted(sizes)
    assert lib.lmoe_w4_experts_workspace_size(1, 16, 896, 3584, 512, None) == INVALID


def test_binding_refuses_host_tensors():
    import sparse_moe_layer_bias_gb300 as lm
    with pytest.raises(TypeError):
        lm.lmoe_balance_loss(torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(TypeError):
        lm.lmoe_w4_quantize(torch.zeros(2, 32, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        lm.lmoe_w4_matvec(torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.bfloat16), 32,
                          torch.zeros(1, 32, dtype=torch.bfloat16))


def test_backward_scores_refuses(lib):
    args = [None, None, 8, None, None, None, None, None, 0, None, None, None, 0, None]
    assert lib.lmoe_backward_scores(*args) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(), INVALID),                       # a valid config: the null weights are what is refused
    (dict(expert_w4=48), INVALID), (dict(expert_w4=-32), INVALID), (dict(expert_fp8=1), SHAPE),
    (dict(with_backward=1), SHAPE), (dict(max_tokens=1025), SHAPE)])
def test_w4_handle_refuses(lib, change, status):
    cfg = binding.LmoeConfig(256, 128, 32, 4, 128, 2, 64, 4.0, 25.0, 1e-6, 64, 0, 0, 0, 32)
    for k, v in change.items():
        setattr(cfg, k, v)
    w, out = binding.LmoeWeights(), ctypes.c_void_p()
    assert lib.lmoe_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(out)) == status


def test_w4_status_refuses(lib):
    assert lib.lmoe_w4_status(None, 0, None) == INVALID
    assert lib.lmoe_w4_selftest_timeout(999, None) == INVALID
    assert lib.lmoe_w4_selftest_timeout(1_000_000_001, None) == INVALID


@pytest.mark.parametrize("n", [(1 << 31) - 1, (1 << 31) - 4095])
def test_w4_matvec_refuses_more_rows_than_it_counts(lib, n):
    assert matvec(lib, n=n, ldy=n) == SHAPE
