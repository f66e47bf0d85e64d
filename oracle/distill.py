"""fp64 numpy oracle of the distillation from a teacher's top logits -- TEST
INFRASTRUCTURE ONLY.

Written from the definition in include/rlk.h (rlk_linear_distill_fwd / _bwd) with
dense teacher rows; pinned by tests/test_distill_oracle.py."""
from __future__ import annotations

import numpy as np


def weights(ids, logits, tau, V, teacher_lse=None):
    """Teacher weights as a dense [T, V] matrix, each row's sum of q log q, and
    which rows hold an id outside [0, V)."""
    T, K = ids.shape
    dense = np.zeros((T, V))
    qlogq = np.zeros(T)
    bad = np.zeros(T, bool)
    for t in range(T):
        slots = [(int(i), float(g) / tau) for i, g in zip(ids[t], logits[t]) if i != -1]
        bad[t] = any(i < 0 or i >= V for i, _ in slots)
        slots = [(i, a) for i, a in slots if 0 <= i < V]
        a = np.array([a for _, a in slots])
        if not slots or (a == -np.inf).all():
            continue
        with np.errstate(invalid="ignore"):
            if teacher_lse is not None:
                L = float(teacher_lse[t])
            else:
                L = a.max() + np.log(np.exp(a - a.max()).sum())
            logq = a - L
        for (i, _), lq in zip(slots, logq):
            q = np.exp(lq)
            dense[t, i] += q
            if q != 0:
                qlogq[t] += q * lq
    return dense, qlogq, bad


def student(hidden, W, tau):
    z = hidden.astype(np.float64) @ W.astype(np.float64).T / tau
    m = z.max(1, keepdims=True)
    lse = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]
    return z, lse


def forward(hidden, W, ids, logits, tau, teacher_tau, teacher_lse=None):
    """(loss, lse) of float64-valued inputs."""
    dense, qlogq, bad = weights(ids, logits, teacher_tau, W.shape[0], teacher_lse)
    z, lse = student(hidden, W, tau)
    loss = qlogq - np.einsum("tv,tv->t", dense, z - lse[:, None])
    return np.where(bad, np.nan, loss), lse


def dlogits(hidden, W, ids, logits, tau, teacher_tau, dloss, teacher_lse=None):
    dense, _, _ = weights(ids, logits, teacher_tau, W.shape[0], teacher_lse)
    z, lse = student(hidden, W, tau)
    p = np.exp(z - lse[:, None])
    return (dloss[:, None] / tau) * (dense.sum(1, keepdims=True) * p - dense)


def backward(hidden, W, ids, logits, tau, teacher_tau, dloss, teacher_lse=None):
    """(dHidden, dW)."""
    dx = dlogits(hidden, W, ids, logits, tau, teacher_tau, dloss, teacher_lse)
    return dx @ W.astype(np.float64), dx.T @ hidden.astype(np.float64)
