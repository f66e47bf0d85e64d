"""Argument checks of rlk_token_probs and rlk_draft_verify that need no GPU: the
pointers here are never dereferenced."""
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
    return binding._samp()


def _probs(L, x=A, xt=F32, R=4, V=100, ldx=100, tau=1.0, rt=None, p=A, pt=F32, ldp=100, ws=W, wsb=256):
    return L.rlk_token_probs(x, xt, R, V, ldx, tau, rt, p, pt, ldp, ws, wsb, None)


def test_probs_argument_errors(L):
    assert L.rlk_sampling_workspace_bytes() == 256
    assert _probs(L, R=-1) == INVALID
    assert _probs(L, V=0) == INVALID
    assert _probs(L, ldx=99) == INVALID
    assert _probs(L, ldp=99) == INVALID
    assert _probs(L, xt=2) == INVALID and _probs(L, pt=-1) == INVALID
    for tau in (-1.0, float("nan"), float("inf"), 1e-45):
        assert _probs(L, tau=tau) == INVALID, tau
    assert _probs(L, V=1 << 31, ldx=1 << 31, ldp=1 << 31) == SHAPE
    assert _probs(L, R=1 << 28) == SHAPE
    assert _probs(L, ldx=1 << 31) == SHAPE
    assert _probs(L, R=0, x=None, p=None) == OK
    for k in ("x", "p", "ws"):
        assert _probs(L, **{k: None}) == INVALID, k
    assert _probs(L, x=A + 2) == MISALIGNED
    assert _probs(L, x=A + 1, xt=BF16) == MISALIGNED
    assert _probs(L, p=A + 2) == MISALIGNED
    assert _probs(L, rt=A + 2) == MISALIGNED
    assert _probs(L, ws=W + 16) == MISALIGNED
    assert _probs(L, wsb=255) == WS_SMALL


def _verify(L, p=A, psb=500, psk=100, q=A, qsb=400, qsk=100, t=F32, d=A, ua=A, us=A, lens=None, B=3, K=4,
            V=100, tok=A, n=A, ws=W, wsb=256):
    return L.rlk_draft_verify(p, psb, psk, q, qsb, qsk, t, d, ua, us, lens, B, K, V, tok, n, ws, wsb, None)


def test_verify_argument_errors(L):
    assert _verify(L, B=-1) == INVALID
    assert _verify(L, K=-1) == INVALID
    assert _verify(L, V=0) == INVALID
    assert _verify(L, t=7) == INVALID
    assert _verify(L, psk=-100) == INVALID and _verify(L, qsb=-1) == INVALID
    assert _verify(L, V=1 << 31) == SHAPE
    assert _verify(L, K=1 << 20) == SHAPE
    assert _verify(L, B=1 << 28) == SHAPE
    assert _verify(L, B=0, p=None) == OK
    for k in ("p", "us", "tok", "n", "ws", "d", "ua"):
        assert _verify(L, **{k: None}) == INVALID, k
    for k in ("p", "q", "us", "ua"):
        assert _verify(L, **{k: A + 2}) == MISALIGNED, k
    for k in ("d", "lens", "tok", "n"):
        assert _verify(L, **{k: A + 4}) == MISALIGNED, k
    assert _verify(L, ws=W + 128) == MISALIGNED
    assert _verify(L, wsb=0) == WS_SMALL


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU refusal")
def test_valid_calls_without_a_gpu_are_refused(L):
    assert _probs(L) == DEVICE
    assert _verify(L) == DEVICE
    assert _verify(L, q=None, lens=A) == DEVICE
    assert _verify(L, K=0, d=None, ua=None, q=None) == DEVICE


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        binding.rlk_token_probs(x)
    with pytest.raises(ValueError):
        binding.rlk_draft_verify(torch.zeros(1, 2, 8), None, torch.zeros(1, 1, dtype=torch.int64),
                                 torch.zeros(1, 1), torch.zeros(1))
