"""The sampling oracle against closed forms and against frequencies: the output
of a verification is distributed as the target whatever the draft is."""
import numpy as np

from oracle import sampling


def test_probs_closed_forms():
    x = np.array([0.0, np.log(3.0), -np.inf])
    assert np.allclose(sampling.token_probs(x, 1.0), [0.25, 0.75, 0.0], atol=1e-15)
    assert np.allclose(sampling.token_probs(x, 0.5), [0.1, 0.9, 0.0], atol=1e-15)
    assert sampling.token_probs(np.array([1.0, 2.0, 2.0]), 0).tolist() == [0, 1, 0]
    assert sampling.token_probs(np.full(3, -np.inf), 1.0).tolist() == [0, 0, 0]
    low = np.finfo(np.float32).min
    assert np.allclose(sampling.token_probs(np.full(4, low), 1.0), 0.25)
    for bad in ([np.nan, 0.0], [np.inf, 0.0]):
        assert np.isnan(sampling.token_probs(np.array(bad), 1.0)).all()
    assert np.isnan(sampling.token_probs(np.zeros(2), -1.0)).all()


def test_draw_by_hand():
    r = np.array([0.0, 0.25, 0.0, 0.5, 0.25, 0.0])
    assert [sampling.draw(r, u) for u in (0.0, 0.24, 0.25, 0.74, 0.75, 0.999, 1.0)] == \
        [1, 1, 3, 3, 4, 4, 4]
    assert sampling.draw(np.zeros(3), 0.5) is None
    assert sampling.draw(np.array([np.nan, 1.0]), 0.5) is None


def test_verify_by_hand():
    p = np.array([[[0.5, 0.5, 0.0], [0.2, 0.3, 0.5], [1.0, 0.0, 0.0]]])
    q = np.array([[[0.25, 0.75, 0.0], [0.9, 0.05, 0.05]]])
    d = np.array([[1, 0]])
    # 0.6 * 0.75 < 0.5; 0.3 * 0.9 > 0.2: rejected, residual (0, 0.25, 0.45)
    tok, n = sampling.draft_verify(p, q, d, np.array([[0.6, 0.3]]), np.array([0.4]))
    assert tok.tolist() == [[1, 2, -1]] and n.tolist() == [1]
    tok, n = sampling.draft_verify(p, q, d, np.array([[0.6, 0.1]]), np.array([0.4]))
    assert tok.tolist() == [[1, 0, 0]] and n.tolist() == [2]
    tok, n = sampling.draft_verify(p, q, d, np.array([[0.6, 0.1]]), np.array([0.4]), [0])
    assert tok.tolist() == [[0, -1, -1]] and n.tolist() == [0]
    # without draft probabilities the draft counts as certain
    tok, n = sampling.draft_verify(p, None, d, np.array([[0.6, 0.1]]), np.array([0.9]))
    assert tok.tolist() == [[0, -1, -1]] and n.tolist() == [0]


def test_first_token_has_the_targets_distribution():
    rng = np.random.default_rng(0)
    V, N = 6, 60000
    p = rng.dirichlet(np.ones(V), 2)
    q = rng.dirichlet(np.ones(V))
    d = rng.choice(V, size=(N, 1), p=q)
    tok, _ = sampling.draft_verify(np.broadcast_to(p, (N, 2, V)), np.broadcast_to(q, (N, 1, V)), d,
                                   rng.random((N, 1)), rng.random(N))
    freq = np.bincount(tok[:, 0], minlength=V) / N
    assert np.all(np.abs(freq - p[0]) < 5 * np.sqrt(p[0] * (1 - p[0]) / N))
