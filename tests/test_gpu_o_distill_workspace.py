"""The distillation's workspaces on the GPU: one for the largest batch serves smaller
ones, to the same bits in either order of the backward; and what LinearDistill keeps
between its passes."""
import pytest
import torch

from invariant_lm_head_gemm_b200 import binding
from tests.test_gpu_n_distill import BF16, F32, _case, _run

pytestmark = pytest.mark.gpu


def _cut(c, n):
    return tuple(t[:n].contiguous() if i != 1 and t is not None else t for i, t in enumerate(c))


@pytest.mark.parametrize("dW_dtype", [F32, BF16, None])
def test_one_workspace_for_several_batches(dW_dtype):
    T, H, V, K = 1024, 4096, 20000, 12
    c = _case(T, H, V, K, 61, std=0.02, tail=True)
    ws = binding.make_distill_workspace(T, H, V, K)
    for n in (512, 1024, 100, 1):
        s = _cut(c, n)
        own = _run(*s, 1.0, 1.0, dW_dtype)
        got = _run(*s, 1.0, 1.0, dW_dtype, ws)
        assert own[4] == 0 and got[4] == 0
        for a, b in zip(got[:4], own[:4]):
            assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("T,H,V", [(3, 64, 20000), (257, 320, 33000), (512, 1024, 50000)])
@pytest.mark.parametrize("dW_dtype", [F32, BF16, None])
def test_both_orders_give_the_same_bits(T, H, V, dW_dtype):
    """A workspace without the few-row order's regions takes the other one; nothing
    behind its end is touched."""
    K = 9
    c = _case(T, H, V, K, 62)

    def a(x):
        return (x + 255) // 256 * 256
    least = binding.workspace_bytes(T, H, V, True) + 3 * a(T * K * 4) + 2 * a(T * 4) + a(T * (-(-V // 256)) * 8)
    full = binding.make_distill_workspace(T, H, V, K)
    assert full.numel() > least
    want = _run(*c, 1.0, 1.0, dW_dtype, full)
    room = torch.full((least + 4096,), 7, dtype=torch.uint8, device="cuda")
    room[:256] = 0
    got = _run(*c, 1.0, 1.0, dW_dtype, room[:least])
    assert got[4] == 0 and (room[least:] == 7).all()
    for x, y in zip(got[:4], want[:4]):
        assert (x is None and y is None) or torch.equal(x, y)
