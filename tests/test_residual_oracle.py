"""Pins of the residual's oracle: the generator's published vectors, a dropout's shares, the norms' closed forms, and
the gradients against differences of the forward form."""
import numpy as np
import pytest

from oracle import residual_oracle as O


def test_generator_vectors():
    # known answers published with the generator: all zeros, all ones, and digits of pi
    assert [hex(v) for v in O.philox([0], 0, 0)[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    ones = (1 << 64) - 1
    assert [hex(v) for v in O.philox([ones], ones, ones)[0]] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]
    got = O.philox([0x85A308D3243F6A88], 0x0370734413198A2E, 0x299F31D0A4093822)[0]
    assert [hex(v) for v in got] == ["0xd16cfe09", "0x94fdcceb", "0x5001e420", "0x24126ea1"]


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_factors(p):
    n = 40000
    f = O.factors(n, p, 1234567, 3)
    kept = (f != 0).mean()
    assert abs(kept - (1 - p)) <= 5 * np.sqrt(p * (1 - p) / n) + 2.0 ** -16  # five deviations
    if p < 1:
        assert np.allclose(f[f != 0], 1 / (1 - p), rtol=2.0 ** -15)
    assert not np.array_equal(O.factors(64, 0.5, 1), O.factors(64, 0.5, 2))
    assert not np.array_equal(O.factors(64, 0.5, 1), O.factors(64, 0.5, 1, 1))


def test_unit_rows():
    y = np.full((2, 8), 3.0)
    ro, x, mag, inv1, inv2 = O.add_norm(y, np.full((2, 8), -1.0), np.ones(8), 2 * np.ones(8), None, 0.5, 0.0)
    assert np.allclose(ro, 0.0) and np.allclose(mag, 2.0) and np.allclose(inv1, 1 / 3)
    ro, x, *_ = O.add_norm(y, y, np.arange(8.0), None, None, 1.0, 0.0)
    assert np.allclose(ro, 6.0) and np.allclose(x, np.arange(8.0))


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gate", ["none", "vector", "full"])
def test_gradients_against_differences(post, pre, gate):
    rng = np.random.default_rng(5)
    N, d = 3, 8
    v = {"y": rng.standard_normal((N, d)), "r": rng.standard_normal((N, d)),
         "w_pre": rng.standard_normal(d) if pre else None, "w_post": rng.standard_normal(d) if post else None,
         "gate": {"none": None, "vector": rng.standard_normal(d), "full": rng.standard_normal((N, d))}[gate]}
    f, eps = 0.7 * O.factors(N * d, 0.3, 9).reshape(N, d), 1e-3
    dx = rng.standard_normal((N, d)) if pre else None
    dro = rng.standard_normal((N, d))

    def loss(v):
        ro, x, *_ = O.add_norm(v["y"], v["r"], v["w_pre"], v["w_post"], v["gate"], f, eps)
        return (ro * dro).sum() + ((x * dx).sum() if pre else 0.0)

    got = O.add_norm_grad(v["y"], v["r"], v["w_pre"], v["w_post"], v["gate"], f, eps, dx, dro)
    of = {"y": "dy", "r": "dr", "w_pre": "dw_pre", "w_post": "dw_post", "gate": "dgate"}
    for name, arr in v.items():
        if arr is None:
            continue
        g = got[of[name]][0]
        g = g.sum(0) if arr.ndim == 1 else g
        h = 1e-5
        for i in np.ndindex(arr.shape):
            up, down = arr.copy(), arr.copy()
            up[i] += h
            down[i] -= h
            diff = (loss({**v, name: up}) - loss({**v, name: down})) / (2 * h)
            # truncation: h^2 / 6 of a third derivative of at most about 1e3 here; rounding: 1e-15 / h
            assert abs(diff - g[i]) <= 1e-6, (name, i)
        assert np.all(np.abs(got[of[name]][0]) <= got[of[name]][1] * (1 + 1e-12))
