"""The chunk-by-chunk order of the distillation's backward over many chunks (three dX
buffers in turn, dHidden added up over the middle chunks), against the formulas in
64 bits on the GPU, with the tolerances that tests/test_gpu_n_distill.py derives."""
import pytest
import torch

from tests import gpu_util as gu
from tests.test_gpu_n_distill import BF16, F32, _case, _run

pytestmark = pytest.mark.gpu

F64 = torch.float64


def _reference(hidden, W, ids, logits, lse, dloss, tau, tau_t):
    """Values and tolerances of loss, dH and dW (all rows' ids inside [0, V))."""
    h, w = hidden.double(), W.double()
    T, H = h.shape
    V = w.shape[0]
    used = ids >= 0
    a = (logits.double() / tau_t).masked_fill(~used, float("-inf"))
    empty = ~(a > float("-inf")).any(1)
    a0 = a.masked_fill(empty[:, None], 0.0)
    logq = (a - lse.double()[:, None]) if lse is not None else a0.log_softmax(1)
    logq = logq.masked_fill(~used | empty[:, None], float("-inf"))
    q = logq.exp()
    z = h @ w.t() / tau
    s = z.logsumexp(1)
    at = ids.clamp(min=0)
    loss = torch.where(q > 0, q * (logq - z.gather(1, at) + s[:, None]), 0.0).sum(1)
    dense = torch.zeros(T, V, dtype=F64, device="cuda").scatter_add_(1, at, q)
    Q = dense.sum(1)
    p = (z - s[:, None]).exp()
    g = dloss.double()
    dx = (g / tau)[:, None] * (Q[:, None] * p - dense)
    ez = (H / 16 + 16) * 2.0 ** -23 * (h.abs() @ w.abs().t()).max(1).values / tau
    big = a.masked_fill(~torch.isfinite(a), 0.0).abs().max(1).values
    la = big + (lse.double().abs() if lse is not None else big + 6)
    ep = 2 * ez + 6e-5 + 2.0 ** -20 * z.abs().max(1).values * 1.4427 + 2.0 ** -20 * la
    slack = 2.0 ** -8 * dx.abs() + (ep * g.abs() / tau)[:, None] * (Q[:, None] * p + dense)
    kh, kt = (V / 16 + 16) * 2.0 ** -23, (T / 16 + 16) * 2.0 ** -23
    return {"loss": (loss, Q * ep + 1e-7),
            "dH": (dx @ w, slack @ w.abs() + kh * (dx.abs() @ w.abs()) + 1e-30),
            "dW": (dx.t() @ h, slack.t() @ h.abs() + kt * (dx.abs().t() @ h.abs()) + 1e-30)}


@pytest.mark.parametrize("T,H,V,tail", [(600, 4096, 33000, True), (300, 8192, 25000, False),
                                        (2100, 1024, 41000, False)])
def test_many_chunks(T, H, V, tail):
    K = 24
    tau, tau_t = (0.8, 1.5) if tail else (1.0, 1.0)
    c = _case(T, H, V, K, T + V, std=1.28 / H ** 0.5, tail=tail, tau_t=tau_t)
    ref = _reference(*c, tau, tau_t)
    runs = {d: _run(*c, tau, tau_t, d) for d in (F32, BF16, None)}
    loss, _, dH, dW, err = runs[F32]
    assert err == 0
    for name, got in (("loss", loss), ("dH", dH), ("dW", dW)):
        want, tol = ref[name]
        step = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -23
        off = (got.double() - want).abs()
        assert (off <= (tol + step * want.abs()) * (1 + 2.0 ** -8)).all(), name
        if name != "loss":
            assert float((got.double() - want).norm() / want.norm()) <= gu.FROB_TOL, name
    assert torch.equal(runs[BF16][3], dW.to(BF16)) and runs[None][3] is None
    for d in (BF16, None):
        assert runs[d][4] == 0
        assert torch.equal(runs[d][0], loss) and torch.equal(runs[d][2], dH)
    again = _run(*c, tau, tau_t, BF16)
    for a, b in zip(again[:4], runs[BF16][:4]):
        assert torch.equal(a, b)
