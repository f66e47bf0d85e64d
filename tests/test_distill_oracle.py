"""The distillation oracle: closed forms, and its gradients against central
differences of its loss."""
import numpy as np
import pytest

from oracle import distill


def _case(T=4, H=6, V=9, K=3, seed=0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.choice(V, K, replace=False) for _ in range(T)])
    return (rng.standard_normal((T, H)), rng.standard_normal((V, H)), ids, rng.standard_normal((T, K)),
            rng.standard_normal(T))


def test_closed_forms():
    hidden, W, ids, logits, _ = _case()
    # one certain slot: the cross entropy of its token
    loss, lse = distill.forward(hidden, W, ids[:, :1], logits[:, :1], 1.0, 1.0)
    z, _ = distill.student(hidden, W, 1.0)
    assert np.allclose(loss, lse - z[np.arange(4), ids[:, 0]])
    # the student's own logits over the whole vocabulary: no loss, no gradient
    every = np.broadcast_to(np.arange(9), (4, 9))
    loss, _ = distill.forward(hidden, W, every, z, 1.0, 1.0)
    assert np.allclose(loss, 0, atol=1e-12)
    dx = distill.dlogits(hidden, W, every, z, 1.0, 1.0, np.ones(4))
    assert np.allclose(dx, 0, atol=1e-12)
    # renormalising is what the slots' own lse does
    L = np.log(np.exp(logits / 2).sum(1))
    a = distill.forward(hidden, W, ids, logits, 0.7, 2.0)[0]
    b = distill.forward(hidden, W, ids, logits, 0.7, 2.0, L)[0]
    assert np.allclose(a, b)


def test_unused_repeated_and_bad_slots():
    hidden, W, ids, logits, g = _case(T=5)
    ids, logits = ids.copy(), logits.copy()
    ids[0] = -1
    logits[0] = np.nan
    ids[1, 2] = -1
    logits[2] = -np.inf
    ids[3] = [4, 4, 2]
    ids[4, 0] = 9
    loss, _ = distill.forward(hidden, W, ids, logits, 1.0, 1.0)
    assert loss[0] == 0 and loss[2] == 0 and np.isnan(loss[4])
    dx = distill.dlogits(hidden, W, ids, logits, 1.0, 1.0, g)
    assert (dx[[0, 2]] == 0).all() and np.isfinite(dx).all()
    assert np.allclose(dx.sum(1), 0)
    two = distill.forward(hidden[1:2], W, ids[1:2, :2], logits[1:2, :2], 1.0, 1.0)[0]
    assert np.allclose(loss[1], two[0])


@pytest.mark.parametrize("tail", [False, True])
def test_gradients_are_those_of_the_loss(tail):
    hidden, W, ids, logits, g = _case(seed=3)
    lse_t = np.log(np.exp(logits).sum(1)) + 0.4 if tail else None

    def total(h, w):
        return (distill.forward(h, w, ids, logits, 0.8, 1.3, lse_t)[0] * g).sum()

    dH, dW = distill.backward(hidden, W, ids, logits, 0.8, 1.3, g, lse_t)
    eps = 1e-6
    for at in np.ndindex(*hidden.shape):
        e = np.zeros_like(hidden)
        e[at] = eps
        assert abs((total(hidden + e, W) - total(hidden - e, W)) / (2 * eps) - dH[at]) < 1e-7
    for at in np.ndindex(*W.shape):
        e = np.zeros_like(W)
        e[at] = eps
        assert abs((total(hidden, W + e) - total(hidden, W - e)) / (2 * eps) - dW[at]) < 1e-7
