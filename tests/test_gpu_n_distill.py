"""Distillation from a teacher's top logits against the fp64 oracle.

Tolerances.  A logit is a dot product of exact bf16 products added in fp32, 16
at a time: |dz| <= (H / 16 + 16) 2^-23 sum |h w| / tau =: e_z, rounding or
truncating.  The lse adds its sum's error: 512 additions of a split, the splits'
merge and the approximate exponentials, below 6e-5 relative; forming y, y - m
and the last products, 8 half steps of the largest |y|.  The loss weighs both by
the q_k, Q in all, with the logarithms of the weights off by a few half steps of
the teacher's scaled logits:
    |dloss| <= Q (2 e_z + 6e-5 + 2^-20 max|y| + 2^-20 (max|a| + |L|)).
A gradient's elements are sums of dlogits that are off by half a step of bf16
(2^-8), by the error of p (2 e_z + 6e-5 + ..., relative) and by that of q; the
result is rounded once more where it is bf16:
    |d dH| <= sum_v (2^-8 |dx_v| + e_p (Q p_v + dense_v) |dloss| / tau) |W_v| + 2^-8 |dH|.
That holds element by element; in the norm, roundings being independent, the
error is about 2^-8 0.42 sqrt(2) = 2.4e-3, and the linear-logp's 5e-3 is held for
cases of many rows."""
import numpy as np
import pytest
import torch

from invariant_lm_head_gemm_b200 import binding
from oracle import distill
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _case(T, H, V, K, seed, std=0.05, teacher=F32, unused=True, tail=False, tau_t=1.0, near=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*n):
        return torch.rand(*n, generator=g, device="cuda")

    def randn(*n):
        return torch.randn(*n, generator=g, device="cuda")

    hidden = randn(T, H).to(BF16)
    W = (std * randn(V, H)).to(BF16)
    kk = min(K, V)
    span = min(V, 40 + kk) if near else V      # near: many ids in one 32-column chunk
    ids = rand(T, span).argsort(1)[:, :kk].contiguous()
    if kk < K:
        ids = torch.cat([ids, ids.new_full((T, K - kk), -1)], 1)
    logits = (2 * randn(T, K)).to(teacher)
    lse = None
    if tail:
        lse = torch.logsumexp(logits.float() / tau_t, 1) + 0.5 * rand(T)
    if unused and T > 3:
        drop = rand(T, K) < 0.3
        drop[1] = True
        ids = ids.masked_fill(drop, -1)
        logits = logits.masked_fill(drop, float("nan"))
        logits[2] = torch.where(torch.isnan(logits[2]), logits[2], float("-inf"))
    return hidden, W, ids, logits, lse, randn(T)


def _f64(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


class _Ref:
    def __init__(self, hidden, W, ids, logits, lse, dloss, tau, tau_t):
        h, w, i, l, L, g = _f64(hidden), _f64(W), ids.cpu().numpy(), _f64(logits), _f64(lse), _f64(dloss)
        H, V = h.shape[1], w.shape[0]
        self.loss, self.lse = distill.forward(h, w, i, l, tau, tau_t, L)
        self.dH, self.dW = distill.backward(h, w, i, l, tau, tau_t, g, L)
        dense, _, self.bad = distill.weights(i, l, tau_t, V, L)
        z, _ = distill.student(h, w, tau)
        ez = (H / 16 + 16) * 2.0 ** -23 * (np.abs(h) @ np.abs(w).T).max(1) / tau
        ymax = np.abs(z).max(1) * 1.4427
        a = np.where((i >= 0) & (i < V), np.nan_to_num(l, nan=0.0, neginf=0.0, posinf=0.0), 0.0) / tau_t
        la = np.abs(a).max(1) + (np.abs(L) if L is not None else np.abs(a).max(1) + 6)
        ep = 2 * ez + 6e-5 + 2.0 ** -20 * ymax + 2.0 ** -20 * la
        Q = dense.sum(1)
        self.tol_loss = Q * ep + 1e-7
        self.tol_lse = ez + 6e-5 + 2.0 ** -20 * ymax
        dx = distill.dlogits(h, w, i, l, tau, tau_t, g, L)
        p = np.exp(z - self.lse[:, None])
        slack = 2.0 ** -8 * np.abs(dx) + (ep * np.abs(g) / tau)[:, None] * (Q[:, None] * p + dense)
        kh, kt = (V / 16 + 16) * 2.0 ** -23, (h.shape[0] / 16 + 16) * 2.0 ** -23
        self.tol_dH = slack @ np.abs(w) + kh * (np.abs(dx) @ np.abs(w)) + 1e-30
        self.tol_dW = slack.T @ np.abs(h) + kt * (np.abs(dx).T @ np.abs(h)) + 1e-30


def _check(ref, loss, lse, dH, dW, frob=True):
    loss, lse = _f64(loss), _f64(lse)
    ok = ~ref.bad
    assert np.isnan(loss[ref.bad]).all()
    assert np.all(np.abs(loss - ref.loss)[ok] <= ref.tol_loss[ok]), np.abs(loss - ref.loss)[ok].max()
    assert np.all(np.abs(lse - ref.lse) <= ref.tol_lse)
    for got, want, tol in ((dH, ref.dH, ref.tol_dH), (dW, ref.dW, ref.tol_dW)):
        if got is None:
            continue
        step = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -23
        got = _f64(got)
        assert np.all(np.abs(got - want) <= tol * (1 + 2.0 ** -8) + step * np.abs(want) * (1 + 2.0 ** -8))
        if frob:
            assert gu.rel_frob(got, want) <= gu.FROB_TOL


def _run(hidden, W, ids, logits, lse, dloss, tau, tau_t, dW_dtype=F32, ws=None):
    T, H = hidden.shape
    if ws is None:
        ws = binding.make_distill_workspace(T, H, W.shape[0], ids.shape[1])
    loss, s = binding.rlk_linear_distill_fwd(hidden, W, ids, logits, tau, tau_t, lse, ws)
    dH, dW = binding.rlk_linear_distill_bwd(hidden, W, ids, logits, tau, s, dloss, tau_t, lse, ws,
                                            dW_dtype=dW_dtype)
    torch.cuda.synchronize()
    return loss, s, dH, dW, binding.rlk_read_device_error(ws)


SHAPES = [
    # T, H, V, K: the short-batch kernel in its forms (a large H and a small vocabulary)
    (1, 4096, 513, 5), (16, 4096, 1500, 8), (32, 4096, 600, 20), (40, 4096, 3000, 33), (130, 4096, 2000, 64),
    (250, 4096, 1100, 16),
    # the pair kernel, ragged vocabularies, chunk borders
    (1, 64, 1, 1), (1, 256, 1000, 1), (2, 64, 31, 8), (16, 128, 513, 20), (17, 64, 700, 5),
    (33, 128, 2000, 64), (64, 256, 1024, 8), (100, 192, 8193, 33), (224, 64, 1537, 100),
    (256, 64, 4097, 256), (257, 64, 1000, 7), (300, 256, 8192, 128), (513, 128, 8500, 32),
    (700, 64, 17000, 16),
    # few rows over several vocabulary chunks
    (1, 64, 8193, 3), (2, 128, 20000, 9), (3, 64, 151936, 40), (257, 320, 16385, 20),
]


@pytest.mark.parametrize("T,H,V,K", SHAPES)
@pytest.mark.parametrize("tail", [False, True])
def test_matches_the_oracle(T, H, V, K, tail):
    tau, tau_t = (0.7, 1.5) if tail else (1.0, 1.0)
    c = _case(T, H, V, K, T + V + K, tail=tail, tau_t=tau_t)
    ref = _Ref(*c, tau, tau_t)
    loss, lse, dH, dW, err = _run(*c, tau, tau_t)
    assert err == 0
    _check(ref, loss, lse, dH, dW, frob=T >= 64)
    if T > 3:  # the rows that _case leaves without a weight
        assert loss[1] == 0 and loss[2] == 0
        assert (dH[1:3] == 0).all()


@pytest.mark.parametrize("T,H", [(5, 64), (40, 64), (129, 64), (600, 64), (7, 4096), (40, 4096), (129, 4096)])
def test_many_ids_in_one_chunk(T, H):
    c = _case(T, H, 3001, 60, T, near=True, unused=False)
    _check(_Ref(*c, 1.0, 1.0), *_run(*c, 1.0, 1.0)[:4], frob=False)


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("dW_dtype", [F32, BF16, None])
def test_dw_types_and_the_frozen_head(T, dW_dtype):
    c = _case(T, 128, 20000, 12, 5, teacher=BF16)
    full = _run(*c, 1.0, 2.0)
    loss, lse, dH, dW, err = _run(*c, 1.0, 2.0, dW_dtype)
    assert err == 0
    assert torch.equal(dH, full[2]) and torch.equal(loss, full[0])
    if dW_dtype is None:
        assert dW is None
    else:
        assert torch.equal(dW, full[3].to(dW_dtype))
    _check(_Ref(*c, 1.0, 2.0), loss, lse, dH, dW)


@pytest.mark.parametrize("T", [3, 50, 250, 400])
@pytest.mark.parametrize("H", [256, 4096])
def test_lse_and_loss_are_those_of_linear_logp(T, H):
    """One certain slot per row is the cross entropy of linear-logp."""
    V = 5000
    hidden, W, ids, _, _, _ = _case(T, H, V, 1, 9, unused=False)
    loss, lse = binding.rlk_linear_distill_fwd(hidden, W, ids, torch.zeros(T, 1, device="cuda"), 0.9)
    logp, _, lse2 = binding.rlk_linear_logp_fwd(hidden, W, ids[:, 0].contiguous(), 0.9)
    assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))
    assert torch.equal(loss, -logp)


@pytest.mark.parametrize("H", [128, 4096])
def test_rows_do_not_depend_on_the_batch_the_place_or_the_order_of_slots(H):
    V, K = 9000, 24
    hidden, W, ids, logits, lse, dloss = _case(600, H, V, K, 21, tail=True)
    full = _run(hidden, W, ids, logits, lse, dloss, 1.0, 1.0)
    again = _run(hidden, W, ids, logits, lse, dloss, 1.0, 1.0)
    for a, b in zip(full[:4], again[:4]):
        assert torch.equal(a, b)
    for lo, hi in ((0, 1), (5, 25), (100, 190), (200, 456), (7, 300)):
        s = slice(lo, hi)
        got = _run(hidden[s].contiguous(), W, ids[s].contiguous(), logits[s].contiguous(),
                   lse[s].contiguous(), dloss[s].contiguous(), 1.0, 1.0)
        assert torch.equal(got[0], full[0][s]) and torch.equal(got[1], full[1][s])
        assert torch.equal(got[2], full[2][s])
    perm = torch.rand(600, K, device="cuda").argsort(1)
    got = _run(hidden, W, ids.gather(1, perm), logits.gather(1, perm), lse, dloss, 1.0, 1.0)
    for a, b in zip(full[:4], got[:4]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [6, 300])
def test_repeated_bad_and_infinite_slots(T):
    H, V, K = 64, 800, 6
    hidden, W, ids, logits, _, dloss = _case(T, H, V, K, 33, unused=False)
    ids[0] = ids[0, :1]                          # one id six times
    ids[1, 2:4] = 799
    ids[2, 0], ids[3, 1], ids[4, 2] = V, -2, 1 << 40
    logits[5, 1] = float("-inf")
    c = (hidden, W, ids, logits, None, dloss)
    ref = _Ref(*c, 1.0, 1.0)
    loss, lse, dH, dW, err = _run(*c, 1.0, 1.0)
    assert err == binding.RLK_DEVERR_TARGET
    assert ref.bad.sum() == 3 and torch.isnan(loss[2:5]).all() and torch.isfinite(dH).all()
    _check(ref, loss, lse, dH, dW, frob=False)
    # a NaN logit, or +inf, in a used slot: that row alone
    logits[0, 0], logits[1, 0] = float("nan"), float("inf")
    ids[2:5] = ids[5:6]
    got = _run(hidden, W, ids, logits, None, dloss, 1.0, 1.0)
    assert torch.isnan(got[0][:2]).all() and torch.isfinite(got[0][2:]).all()
    assert torch.isnan(got[2][:2]).any(1).all() and torch.isfinite(got[2][2:]).all()


def test_gradient_against_differences():
    """The forward's own loss, stepped along the gradient's direction."""
    T, H, V, K = 300, 256, 3000, 16
    hidden, W, ids, logits, lse, _ = _case(T, H, V, K, 44, std=0.02, tail=True)
    dloss = torch.ones(T, device="cuda")
    loss, s, dH, dW, _ = _run(hidden, W, ids, logits, lse, dloss, 1.0, 1.0)
    d = dH.double() / dH.double().norm()
    step = 4.0
    up = (hidden.double() + step * d).to(BF16)
    down = (hidden.double() - step * d).to(BF16)
    a = binding.rlk_linear_distill_fwd(up, W, ids, logits, 1.0, teacher_lse=lse)[0].double().sum()
    b = binding.rlk_linear_distill_fwd(down, W, ids, logits, 1.0, teacher_lse=lse)[0].double().sum()
    # what the rounded steps really were, along the gradient
    want = (dH.double() * (up.double() - down.double())).sum()
    assert abs((a - b) - want) <= 0.02 * abs(want)


def test_empty_batch_and_refusals():
    hidden, W, ids, logits, _, dloss = _case(4, 64, 300, 3, 2)
    e = slice(0, 0)
    loss, lse = binding.rlk_linear_distill_fwd(hidden[e], W, ids[e], logits[e])
    assert loss.shape == (0,) and lse.shape == (0,)
    for dt in (F32, BF16):
        out = (torch.empty(0, 64, dtype=BF16, device="cuda"), torch.full((300, 64), 3.0, dtype=dt, device="cuda"))
        binding.rlk_linear_distill_bwd(hidden[e], W, ids[e], logits[e], 1.0, lse, dloss[e], out=out, dW_dtype=dt)
        assert (out[1] == 0).all()
    for bad in (lambda: binding.rlk_linear_distill_fwd(hidden.float(), W, ids, logits),
                lambda: binding.rlk_linear_distill_fwd(hidden, W[:, :32], ids, logits),
                lambda: binding.rlk_linear_distill_fwd(hidden, W, ids.int(), logits),
                lambda: binding.rlk_linear_distill_fwd(hidden, W, ids[:, :2], logits),
                lambda: binding.rlk_linear_distill_fwd(hidden, W, ids, logits.double()),
                lambda: binding.rlk_linear_distill_fwd(hidden, W, ids, logits, teacher_lse=dloss[:2]),
                lambda: binding.rlk_linear_distill_fwd(hidden, W, ids[:, :0], logits[:, :0]),
                lambda: binding.rlk_linear_distill_fwd(hidden, W, ids.cpu(), logits),
                lambda: binding.rlk_linear_distill_bwd(hidden, W, ids, logits, 1.0, dloss, dloss.double()),
                lambda: binding.rlk_linear_distill_bwd(hidden, W, ids, logits, 1.0, dloss, dloss,
                                                       dW_dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    small = binding.make_distill_workspace(4, 64, 300, 3, False)
    with pytest.raises(binding.RlkError):
        binding.rlk_linear_distill_bwd(hidden, W, ids, logits, 1.0, dloss, dloss, workspace=small)
    for tau in (0.0, -1.0, float("nan")):
        with pytest.raises(binding.RlkError):
            binding.rlk_linear_distill_fwd(hidden, W, ids, logits, tau)
        with pytest.raises(binding.RlkError):
            binding.rlk_linear_distill_fwd(hidden, W, ids, logits, 1.0, tau)


@pytest.mark.parametrize("frozen", [False, True])
def test_autograd(frozen):
    T, H, V, K = 90, 128, 6000, 10
    hidden, W, ids, logits, lse, _ = _case(T, H, V, K, 55, tail=True)
    h = hidden.clone().requires_grad_(True)
    w = W.clone().requires_grad_(not frozen)
    loss = binding.LinearDistill.apply(h, w, ids, logits, 1.0, None, lse)
    loss.mean().backward()                        # an expanded upstream gradient
    want = _run(hidden, W, ids, logits, lse, torch.full((T,), 1.0 / T, device="cuda"), 1.0, 1.0,
                None if frozen else BF16)
    assert torch.equal(loss.detach(), want[0]) and torch.equal(h.grad, want[2])
    assert w.grad is None if frozen else torch.equal(w.grad, want[3])
    # a head used twice sums its gradients
    if not frozen:
        h2, w2 = hidden.clone().requires_grad_(True), W.clone().requires_grad_(True)
        (binding.LinearDistill.apply(h2, w2, ids, logits, 1.0, None, lse).mean() +
         binding.LinearDistill.apply(h2, w2, ids, logits, 1.0, None, lse).mean()).backward()
        assert torch.equal(w2.grad, w.grad + w.grad)


def test_autograd_without_and_with_one_gradient():
    T, H, V, K = 40, 64, 9000, 6
    hidden, W, ids, logits, lse, _ = _case(T, H, V, K, 56, tail=True)
    want = _run(hidden, W, ids, logits, lse, torch.ones(T, device="cuda"), 1.0, 1.0, BF16)
    with torch.no_grad():
        loss = binding.LinearDistill.apply(hidden.requires_grad_(True), W, ids, logits, 1.0, None, lse)
    assert not loss.requires_grad and torch.equal(loss, want[0])
    w = W.clone().requires_grad_(True)
    loss = binding.LinearDistill.apply(hidden.detach(), w, ids, logits, 1.0, None, lse)
    loss.backward(torch.ones(1, device="cuda").expand(T), retain_graph=True)
    assert torch.equal(w.grad, want[3])
    loss.sum().backward()                          # the saved workspace serves a second pass
    assert torch.equal(w.grad, want[3] + want[3])


@pytest.mark.parametrize("T", [20, 300])
def test_capture_and_side_stream(T):
    H, V, K = 64, 9000, 8
    hidden, W, ids, logits, lse, dloss = _case(T, H, V, K, 66)
    ws = binding.make_distill_workspace(T, H, V, K)
    want = _run(hidden, W, ids, logits, lse, dloss, 1.0, 1.0, BF16)
    fo = (torch.empty(T, device="cuda"), torch.empty(T, device="cuda"))
    bo = (torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(V, H, dtype=BF16, device="cuda"))

    def step(stream=None):
        binding.rlk_linear_distill_fwd(hidden, W, ids, logits, 1.0, teacher_lse=lse, workspace=ws, out=fo,
                                       stream=stream)
        binding.rlk_linear_distill_bwd(hidden, W, ids, logits, 1.0, fo[1], dloss, teacher_lse=lse,
                                       workspace=ws, out=bo, dW_dtype=BF16, stream=stream)

    def check():
        for a, b in zip(fo + bo, want):
            assert torch.equal(a, b)
            a.zero_()

    step()
    torch.cuda.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    check()
    # without a workspace the call's own belongs to its stream
    side.wait_stream(torch.cuda.current_stream())
    loss, _ = binding.rlk_linear_distill_fwd(hidden, W, ids, logits, 1.0, teacher_lse=lse, stream=side)
    side.synchronize()
    assert torch.equal(loss, want[0])


def test_two_streams_at_once():
    """Calls that overlap on the GPU, each with its own workspace (and, for the
    sampling calls, one between them)."""
    cases = [_case(T, 256, 20000, 12, 80 + T, tail=True) for T in (60, 700)]
    want = [_run(*c, 1.0, 1.0, BF16) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [binding.make_distill_workspace(c[0].shape[0], 256, 20000, 12) for c in cases]
    shared = binding.sampling_workspace()
    x = torch.randn(50, 20000, device="cuda")
    p = binding.rlk_token_probs(x, 1.0)
    torch.cuda.synchronize()
    got = [None, None]
    probs = [None, None]
    for _ in range(4):
        for i, (c, st) in enumerate(zip(cases, streams)):
            hidden, W, ids, logits, lse, dloss = c
            loss, s = binding.rlk_linear_distill_fwd(hidden, W, ids, logits, 1.0, teacher_lse=lse,
                                                     workspace=spaces[i], stream=st)
            got[i] = (loss, s) + binding.rlk_linear_distill_bwd(
                hidden, W, ids, logits, 1.0, s, dloss, teacher_lse=lse, workspace=spaces[i],
                dW_dtype=BF16, stream=st)
            probs[i] = binding.rlk_token_probs(x, 1.0, workspace=shared, stream=st)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for u, v in zip(a, b):
            assert torch.equal(u, v)
    assert all(torch.equal(q, p) for q in probs)
    assert all(binding.rlk_read_device_error(w) == 0 for w in spaces + [shared])


@pytest.mark.parametrize("T,H,V,K", [(19, 64, 513, 5), (250, 128, 9000, 40), (300, 64, 8500, 33)])
def test_nothing_is_written_outside(T, H, V, K):
    from tests.test_gpu_k_guard import Guarded
    hidden, W, ids, logits, lse, dloss = _case(T, H, V, K, 71)
    want = _run(hidden, W, ids, logits, lse, dloss, 1.0, 1.0, BF16)
    n = binding.make_distill_workspace(T, H, V, K).numel()
    gw = Guarded(n + 256)
    gl, gs, gh, gd = Guarded(T * 4), Guarded(T * 4), Guarded(T * H * 2), Guarded(V * H * 2)
    raw = gw.view(torch.uint8, n + 256)
    off = -raw.data_ptr() % 256
    ws = raw[off:off + n]
    ws[:256] = 0
    loss, s = gl.view(F32, T), gs.view(F32, T)
    dH, dW = gh.view(BF16, T, H), gd.view(BF16, V, H)
    binding.rlk_linear_distill_fwd(hidden, W, ids, logits, 1.0, teacher_lse=lse, workspace=ws, out=(loss, s))
    binding.rlk_linear_distill_bwd(hidden, W, ids, logits, 1.0, s, dloss, teacher_lse=lse, workspace=ws,
                                   out=(dH, dW), dW_dtype=BF16)
    torch.cuda.synchronize()
    for a, b in zip((loss, s, dH, dW), want):
        assert torch.equal(a, b)
    assert all(g.intact() for g in (gw, gl, gs, gh, gd))


def test_draft_training_and_verification_together():
    """A target's head gives a teacher's top logits; a student's hidden states take
    distillation steps through the same frozen head; the student drafts, and the
    drafts are verified against the target."""
    B, K, H, V, top = 8, 4, 256, 4096, 32
    g = torch.Generator(device="cuda").manual_seed(5)
    W = (0.08 * torch.randn(V, H, generator=g, device="cuda")).to(BF16)
    target = torch.randn(B * (K + 1), H, generator=g, device="cuda").to(BF16)
    student = torch.randn(B * (K + 1), H, generator=g, device="cuda").to(BF16)
    zt, _ = binding.rlk_gemm_bf16_f32(target, W)
    logits, ids = zt.topk(top, dim=1)
    h = student.clone().requires_grad_(True)
    binding.LinearDistill.apply(h, W, ids, logits, 1.0, None, torch.logsumexp(zt, 1)).sum().backward()
    q_dense, _, _ = distill.weights(ids.cpu().numpy(), _f64(logits), 1.0, V,
                                    _f64(torch.logsumexp(zt, 1)))
    z = _f64(student) @ _f64(W).T
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    want = (q_dense.sum(1, keepdims=True) * p - q_dense) @ _f64(W)
    assert gu.rel_frob(_f64(h.grad), want) <= gu.FROB_TOL
    stepped = (student.float() - 8.0 * h.grad.float()).to(BF16)
    zs, _ = binding.rlk_gemm_bf16_f32(stepped, W)
    pt = binding.rlk_token_probs(zt.view(B, K + 1, V), 1.0)
    ps = binding.rlk_token_probs(zs.view(B, K + 1, V)[:, :K].contiguous(), 1.0)
    drafts = (ps / torch.empty_like(ps).exponential_(generator=g)).argmax(-1)
    ua = torch.rand(B, K, generator=g, device="cuda")
    us = torch.rand(B, generator=g, device="cuda")
    tokens, n = binding.rlk_draft_verify(pt, ps, drafts, ua, us)
    from oracle import sampling
    tok, acc = sampling.draft_verify(_f64(pt), _f64(ps), drafts.cpu().numpy(), _f64(ua), _f64(us))
    assert np.array_equal(tokens.cpu().numpy(), tok) and np.array_equal(n.cpu().numpy(), acc)
