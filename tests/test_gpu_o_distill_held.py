"""What LinearDistill holds from its forward to its backward, and its capture."""
import pytest
import torch

from invariant_lm_head_gemm_b200 import binding
from tests.test_gpu_n_distill import _case, _run, BF16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,V", [(512, 256, 60000), (5, 64, 300)])
def test_no_large_workspace_is_held_between_the_passes(T, H, V):
    K = 6
    hidden, W, ids, logits, _, _ = _case(T, H, V, K, 63)
    want = _run(hidden, W, ids, logits, None, torch.ones(T, device="cuda"), 1.0, 1.0, BF16)
    h, w = hidden.clone().requires_grad_(True), W.clone().requires_grad_(True)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    losses = [binding.LinearDistill.apply(h, w, ids, logits) for _ in range(3)]
    held = torch.cuda.memory_allocated() - before
    assert held <= 3 * (1 << 20), held
    sum(loss.sum() for loss in losses).backward()
    assert torch.equal(losses[0].detach(), want[0])
    assert torch.equal(h.grad, (want[2] + want[2]) + want[2])
    assert torch.equal(w.grad, (want[3] + want[3]) + want[3])


@pytest.mark.parametrize("T,H,V", [(70, 128, 20000), (5, 64, 300)])
def test_captured_step(T, H, V):
    """A captured step allocates from the graph's own memory and replays to the
    same bits."""
    K = 6
    hidden, W, ids, logits, _, _ = _case(T, H, V, K, 64)
    h, w = hidden.clone().requires_grad_(True), W.clone().requires_grad_(True)

    def step():
        loss = binding.LinearDistill.apply(h, w, ids, logits)
        return (loss,) + torch.autograd.grad(loss.sum(), (h, w))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.detach().clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.detach(), b)
            a.detach().zero_()
