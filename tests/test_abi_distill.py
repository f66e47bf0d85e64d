"""Argument checks of the distillation that need no GPU (the pointers are never
dereferenced), its workspace sizes and its backward's unit count."""
import pytest
import torch

from invariant_lm_head_gemm_b200 import binding, build

OK, INVALID, SHAPE, MISALIGNED, WS_SMALL, DEVICE, CUDA = range(7)
A = 0x10000
W = 0x20000
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding._dis()


def _fwd(L, h=A, w=A, ids=A, g=A, gt=F32, tl=None, T=4, H=64, V=100, K=8, tau=1.0, tt=1.0, loss=A, lse=A,
         ws=W, wsb=1 << 30):
    return L.rlk_linear_distill_fwd(h, w, ids, g, gt, tl, T, H, V, K, tau, tt, loss, lse, ws, wsb, None)


def _bwd(L, h=A, w=A, ids=A, g=A, gt=F32, tl=None, T=4, H=64, V=100, K=8, tau=1.0, tt=1.0, lse=A, dl=A, dh=A,
         dw=A, dwt=F32, ws=W, wsb=1 << 30):
    return L.rlk_linear_distill_bwd(h, w, ids, g, gt, tl, T, H, V, K, tau, tt, lse, dl, dh, dw, dwt, ws, wsb,
                                    None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_argument_errors(L, call):
    assert call(L, T=-1) == INVALID
    assert call(L, K=0) == INVALID
    assert call(L, K=257) == SHAPE
    assert call(L, H=96) == SHAPE
    assert call(L, V=1 << 31) == SHAPE
    assert call(L, gt=3) == INVALID
    for tau in (0.0, -1.0, float("nan"), float("inf")):
        assert call(L, tau=tau) == INVALID, tau
        assert call(L, tt=tau) == INVALID, tau
    assert call(L, tt=1e-45) == INVALID            # 1 / tt overflows
    for k in ("h", "w", "ids", "g", "lse", "ws"):
        assert call(L, **{k: None}) == INVALID, k
    for k, off in (("h", 8), ("w", 2), ("ids", 4), ("g", 2), ("tl", 2), ("lse", 2)):
        assert call(L, **{k: A + off}) == MISALIGNED, k
    assert call(L, ws=W + 64) == MISALIGNED
    need = L.rlk_linear_distill_workspace_bytes(4, 64, 100, 8, 0 if call is _fwd else 1)
    if call is _fwd:
        assert call(L, wsb=need - 1) == WS_SMALL
    else:
        assert call(L, wsb=need // 2) == WS_SMALL


def test_forward_and_backward_specifics(L):
    assert _fwd(L, loss=None) == INVALID
    assert _fwd(L, T=0, h=None) == OK
    assert _bwd(L, dl=None) == INVALID and _bwd(L, dh=None) == INVALID
    assert _bwd(L, dwt=5) == INVALID
    assert _bwd(L, dw=A + 8) == MISALIGNED and _bwd(L, dh=A + 8) == MISALIGNED


def test_workspace_bytes(L):
    f = L.rlk_linear_distill_workspace_bytes
    assert f(4, 64, 100, 0, 0) == 0 and f(4, 64, 100, 257, 1) == 0 and f(4, 65, 100, 8, 1) == 0
    T, H, V, K = 5980, 4096, 151936, 64

    def a(x):
        return (x + 255) // 256 * 256
    rows = 3 * a(T * K * 4) + 2 * a(T * 4)
    assert f(T, H, V, K, 0) == binding.workspace_bytes(T, H, V, False) + rows + a(T * 297 * 8)
    assert f(T, H, V, K, 1) == binding.workspace_bytes(T, H, V, True) + rows + a(T * 594 * 8)
    assert f(1, 64, 1, 1, 1) >= f(1, 64, 1, 1, 0) > 256


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU refusal")
def test_valid_calls_without_a_gpu_are_refused(L):
    assert _fwd(L) == DEVICE
    assert _fwd(L, gt=BF16, tl=A) == DEVICE
    assert _bwd(L) == DEVICE
    assert _bwd(L, dw=None) == DEVICE
    assert _bwd(L, T=0) == DEVICE


def test_binding_refuses_host_tensors():
    z = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.rlk_linear_distill_fwd(z, z, torch.zeros(2, 1, dtype=torch.int64), torch.zeros(2, 1))
