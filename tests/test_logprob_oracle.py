"""Pins of the log-probabilities' oracle: closed forms, and the gradient against differences."""
import numpy as np

from oracle import logprob_oracle as O


def test_uniform_rows():
    z = np.full((2, 8), 3.0)
    z[1, 4:] = -np.inf
    M, L, H, p, logp = O.row_stats(z)
    assert np.allclose(M, 3.0) and np.allclose(L, [np.log(8), np.log(4)]) and np.allclose(H, L)
    assert np.allclose(p[0], 1 / 8) and np.allclose(p[1], [0.25] * 4 + [0] * 4) and logp[1, 5] == -np.inf
    assert np.allclose(O.given(logp, np.array([[0, -1, 8], [3, 2, 2]])), [[-np.log(8), 0, 0], [-np.log(4)] * 3])


def test_one_token_and_none():
    z = np.full((3, 5), -np.inf)
    z[0, 2] = 7.0
    z[2] = -3.4e38  # all at the type's lowest value: uniform
    M, L, H, p, logp = O.row_stats(z)
    assert H[0] == 0 and p[0, 2] == 1 and logp[0, 2] == 0
    assert M[1] == -np.inf and H[1] == 0 and not p[1].any() and np.all(logp[1] == -np.inf)
    assert np.allclose(H[2], np.log(5))


def test_top_order():
    z = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0, np.nan]])
    ids, lp = O.top(z, z - 5.0, 6)
    assert ids.tolist() == [[1, 2, 4, 0, -1, -1]] and lp[0, 4] == -np.inf and lp[0, 0] == -2.0


def test_gradient_against_differences():
    rng = np.random.default_rng(1)
    N, V, T = 4, 9, 3
    z = 2 * rng.standard_normal((N, V))
    z[1, 3] = -np.inf
    ids = rng.integers(-1, V + 1, (N, T))
    ids[2, 1] = ids[2, 0] = 5  # the same token twice
    w, u = rng.standard_normal((N, T)), rng.standard_normal(N)
    G = O.logits_grad(z, ids, w, u)

    def f(z):
        M, L, H, _, logp = O.row_stats(z)
        held = np.maximum(z, -1e3) - (M + L)[:, None]  # a banned token's logit is held, not its log-probability
        return (w * O.given(held, ids)).sum() + (u * H).sum()

    h = 1e-5
    for i in np.ndindex(z.shape):
        if z[i] == -np.inf:
            # a banned token's logit moves nothing but its own log-probability
            assert G[i] == O.weights(ids, w, V, N)[i]
            continue
        a, b = z.copy(), z.copy()
        a[i] += h
        b[i] -= h
        # truncation below h^2 / 6 x 100, rounding 1e-15 x 1e3 / h
        assert abs((f(a) - f(b)) / (2 * h) - G[i]) <= 1e-6
    assert not O.logits_grad(np.full((1, 3), -np.inf), None, None, np.ones(1)).any()
