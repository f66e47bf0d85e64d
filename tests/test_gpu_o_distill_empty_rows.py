"""Rows that carry no weight give no gradient, whatever stands in their dloss (a mean
over no slots divides by zero): they are zero in dHidden and absent from dW."""
import pytest
import torch

from tests.test_gpu_n_distill import BF16, F32, _case, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,V", [(9, 64, 700), (300, 128, 9000), (600, 4096, 20000)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_dloss_of_rows_without_weight(T, H, V, value):
    hidden, W, ids, logits, lse, dloss = _case(T, H, V, 6, 17, std=0.02, tail=True)
    ids[4] = -1
    ids[5] = V                                     # no slot that counts, though a bad one
    dloss[[1, 2, 4, 5]] = 0.0
    for dW_dtype, L in ((F32, lse), (BF16, None)):
        want = _run(hidden, W, ids, logits, L, dloss, 1.0, 1.0, dW_dtype)
        bad = dloss.clone()
        bad[[1, 2, 4, 5]] = value
        got = _run(hidden, W, ids, logits, L, bad, 1.0, 1.0, dW_dtype)
        assert (got[2][[1, 2, 4, 5]] == 0).all() and torch.isfinite(got[3]).all()
        assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
