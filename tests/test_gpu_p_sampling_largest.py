"""rlk_token_probs and rlk_draft_verify at the largest sizes they take: a row of 2^31 - 1
entries, and sequences of hundreds of thousands of drafts."""
import pytest
import torch

from invariant_lm_head_gemm_b200 import binding
from tests.test_gpu_m_sampling import BF16

pytestmark = pytest.mark.gpu

V = (1 << 31) - 1


def test_probs_of_the_longest_row():
    x = torch.full((1, V), float("-inf"), dtype=BF16, device="cuda")
    at = [0, 1 << 30, V - 2, V - 1]
    x[0, at] = torch.tensor([1.0, 1.0, 0.0, 1.0], dtype=BF16, device="cuda")
    ws = binding.sampling_workspace()
    greedy = torch.empty_like(x)
    binding.rlk_token_probs(x, 0.0, out=greedy, workspace=ws)
    assert float(greedy[0, 0]) == 1 and int((greedy != 0).sum()) == 1
    del greedy
    binding.rlk_token_probs(x, 0.5, out=x, workspace=ws)
    e = torch.tensor([0.0, 0.0, -2.0, 0.0], dtype=torch.float64).exp()
    got = x[0, at].double().cpu()
    assert ((got - e / e.sum()).abs() <= 2.0 ** -7 * e / e.sum()).all()
    assert int((x != 0).sum()) == 4 and binding.rlk_read_device_error(ws) == 0


def test_verify_the_longest_row():
    p = torch.zeros(1, 1, V, dtype=BF16, device="cuda")
    p[0, 0, [0, 1 << 30, V - 1]] = torch.tensor([0.25, 0.25, 0.5], dtype=BF16, device="cuda")
    none = torch.zeros(1, 0, device="cuda")
    for u, token in ((0.1, 0), (0.3, 1 << 30), (0.9, V - 1)):
        tok, n = binding.rlk_draft_verify(p, None, none.long(), none, torch.full((1,), u, device="cuda"))
        assert tok.tolist() == [[token]] and n.tolist() == [0]
    # refused drafts at both ends, with and without the draft's distribution
    q = torch.zeros_like(p)
    q[0, 0, V - 1] = 1.0
    both = p.expand(1, 2, V)
    one, half = torch.full((1, 1), 1.0, device="cuda"), torch.full((1,), 0.6, device="cuda")
    last = torch.full((1, 1), V - 1, device="cuda")
    for draft in (q, None):
        tok, n = binding.rlk_draft_verify(both, draft, last, one, half)
        assert tok.tolist() == [[1 << 30, -1]] and n.tolist() == [0]
    tok, n = binding.rlk_draft_verify(both, q, last, one * 0.25, half)
    assert tok.tolist() == [[V - 1, V - 1]] and n.tolist() == [1]


def test_very_many_drafts():
    K, v = 300001, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    p = torch.rand(2, K + 1, v, generator=g, device="cuda") + 0.5
    d = torch.randint(0, v, (2, K), generator=g, device="cuda")
    ua = torch.zeros(2, K, device="cuda")
    ua[1, K - 7] = 1e9
    q = torch.ones(2, K, v, device="cuda")
    tok, n = binding.rlk_draft_verify(p, q, d, ua, torch.zeros(2, device="cuda"))
    assert n.tolist() == [K, K - 7]
    assert torch.equal(tok[0, :K], d[0]) and int(tok[0, K]) == 0
    assert torch.equal(tok[1, :K - 7], d[1, :K - 7]) and (tok[1, K - 6:] == -1).all()
    r = (p[1, K - 7] - 1.0).clamp(min=0)
    assert int(tok[1, K - 7]) == int((r > 0).nonzero()[0])
