"""fp64 numpy oracle of the rollout-side operators: probabilities of a row of
logits, and the verification of drafted tokens -- TEST INFRASTRUCTURE ONLY.

Written from the definitions in include/rlk.h (rlk_token_probs,
rlk_draft_verify); pinned by tests/test_sampling_oracle.py."""
from __future__ import annotations

import numpy as np


def token_probs(x, tau):
    """softmax(x / tau) of one row; one-hot at the first maximum for tau = 0;
    zeros for a row of -inf; NaN where there is no distribution."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or not (tau >= 0 and np.isfinite(tau)):
        return np.full(x.shape, np.nan)
    if not (x > -np.inf).any():
        return np.zeros(x.shape)
    if tau == 0:
        p = np.zeros(x.shape)
        p[int(np.argmax(x))] = 1.0
        return p
    if (x == np.inf).any():
        return np.full(x.shape, np.nan)
    e = np.exp((x - x.max()) / float(tau))
    return e / e.sum()


def draw(r, u):
    """The least v whose running sum exceeds u times the whole sum; the last v of
    positive r when none does.  None when r gives no distribution."""
    total = r.sum()
    if not (np.isfinite(total) and total > 0):
        return None
    over = np.nonzero(np.cumsum(r) > u * total)[0]
    if u < 1 and over.size:
        return int(over[0])
    return int(np.nonzero(r > 0)[0][-1])


def draft_verify(p, q, drafts, u_accept, u_sample, lens=None):
    """tokens [B, K+1] and accepted counts [B], one sequence and one draft at a
    time.  p [B, K+1, V], q [B, K, V] or None."""
    p = np.asarray(p, np.float64)
    B, K1, V = p.shape
    tokens = np.full((B, K1), -1, np.int64)
    accepted = np.zeros(B, np.int64)
    for b in range(B):
        n = K1 - 1 if lens is None else min(max(int(lens[b]), 0), K1 - 1)
        length = n
        for i in range(length):
            d = int(drafts[b, i])
            if 0 <= d < V:
                qd = 1.0 if q is None else float(q[b, i, d])
                if float(u_accept[b, i]) * qd < p[b, i, d]:
                    tokens[b, i] = d
                    continue
            n = i
            break
        accepted[b] = n
        r = p[b, n]
        with np.errstate(invalid="ignore"):
            if n < length:
                if q is not None:
                    r = r - np.asarray(q[b, n], np.float64)
                    if not np.isfinite(r).all():
                        r = np.full(V, np.nan)
                else:
                    r = r - (np.arange(V) == int(drafts[b, n]))
            r = np.where(r < 0, 0.0, r)
            if n < length and r.sum() == 0:
                r = np.where(p[b, n] < 0, 0.0, p[b, n])
        v = draw(r, float(u_sample[b]))
        tokens[b, n] = -1 if v is None else v
    return tokens, accepted
