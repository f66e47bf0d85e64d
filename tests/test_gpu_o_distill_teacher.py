"""A teacher's row far from zero: without the teacher's own log-sum-exp only the
differences of a row's logits count, so a row and the same row moved by a constant
(both exactly representable) give the same bits, and the moved row keeps the
tolerance of the one at zero (tests/test_gpu_n_distill.py)."""
import pytest
import torch

from tests.test_gpu_n_distill import BF16, F32, _case, _check, _Ref, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("teacher,shift", [(F32, 4096.0), (F32, -65536.0), (F32, 2.0 ** 22), (BF16, 256.0)])
@pytest.mark.parametrize("tau_t", [1.0, 0.7])
@pytest.mark.parametrize("T", [20, 300])
def test_only_differences_of_teacher_logits_count(teacher, shift, tau_t, T):
    H, V, K = 64, 9000, 12
    hidden, W, ids, logits, _, dloss = _case(T, H, V, K, 91, teacher=teacher)
    base = (logits / 2).round() * 2                # even numbers, -inf and NaN as they were
    moved = base + shift
    exact = torch.isfinite(base.float())
    assert torch.equal((moved.double() - shift)[exact], base.double()[exact]) and exact.any(1).sum() > T // 2
    want = _run(hidden, W, ids, base, None, dloss, 1.0, tau_t)
    got = _run(hidden, W, ids, moved, None, dloss, 1.0, tau_t)
    assert got[4] == 0
    _check(_Ref(hidden, W, ids, base, None, dloss, 1.0, tau_t), *got[:4], frob=False)
    for a, b in zip(got[:4], want[:4]):
        assert torch.equal(a, b)


def test_teacher_logits_at_the_ends_of_their_range():
    """Differences past the type's range weigh nothing; small temperatures do not overflow."""
    T, H, V, K = 8, 64, 500, 4
    hidden, W, ids, _, _, dloss = _case(T, H, V, K, 92, unused=False)
    logits = torch.tensor([3e38, -3e38, 3e38, float("-inf")], device="cuda").repeat(T, 1)
    same = torch.tensor([0.0, float("-inf"), 0.0, float("-inf")], device="cuda").repeat(T, 1)
    want = _run(hidden, W, ids, same, None, dloss, 1.0, 1.0)
    for tau_t in (1.0, 1e-30):
        got = _run(hidden, W, ids, logits, None, dloss, 1.0, tau_t)
        assert got[4] == 0 and torch.isfinite(got[0]).all()
        for a, b in zip(got[:4], want[:4]):
            assert torch.equal(a, b)
