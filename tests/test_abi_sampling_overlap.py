"""Outputs laid over inputs, refused before anything runs (no GPU needed; the pointers
are never dereferenced)."""
import pytest
import torch

from tests.test_abi_sampling import A, BF16, DEVICE, F32, INVALID, L, _probs, _verify  # noqa: F401

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="pointers are not real")


def test_probs_in_place_takes_equal_types_and_strides(L):  # noqa: F811
    for t in (BF16, F32):
        assert _probs(L, x=A, p=A, xt=t, pt=t) == DEVICE
        assert _probs(L, x=A, p=A, xt=t, pt=t, ldx=128, ldp=128) == DEVICE
        assert _probs(L, x=A, p=A, xt=t, pt=t, R=1, ldx=128, ldp=100) == DEVICE
        assert _probs(L, x=A, p=A, xt=t, pt=t, ldx=128, ldp=100) == INVALID
        assert _probs(L, x=A, p=A, xt=t, pt=BF16 + F32 - t) == INVALID
        assert _probs(L, x=A, p=A, xt=t, pt=BF16 + F32 - t, R=1) == INVALID
        assert _probs(L, x=A, p=2 * A, xt=t, pt=BF16 + F32 - t) == DEVICE
