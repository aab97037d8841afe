"""Pins of the vocabulary-end oracles against facts fixed by mathematics (CPU)."""
import numpy as np
import pytest

from oracle import vocab_oracle as O


def test_embed_grad_is_the_transpose_of_embed():
    # <dY, embed(W)> = <embed_grad(dY), W> for every W: the gradient is the
    # lookup's transpose, also with repeated and absent tokens
    rng = np.random.default_rng(0)
    ids = np.array([3, -1, 0, 3, 7, 3, 9, 100])
    W, dY = rng.standard_normal((8, 5)), rng.standard_normal((8, 5))
    g, mag, count = O.embed_grad(ids, dY, 8, 2.5)
    assert np.isclose(np.sum(dY * O.embed_rows(ids, W, 2.5)), np.sum(g * W))
    assert count.tolist() == [1, 0, 0, 3, 0, 0, 0, 1]
    assert np.all(mag >= np.abs(g) - 1e-12)


def test_embed_grad_by_differences():
    rng = np.random.default_rng(1)
    ids = np.array([1, 1, 2, 0])
    W, dY = rng.standard_normal((3, 2)), rng.standard_normal((4, 2))
    g, _, _ = O.embed_grad(ids, dY, 3, 0.5)
    for v in range(3):
        for j in range(2):
            E = np.zeros_like(W)
            E[v, j] = 1e-3
            d = np.sum(dY * (O.embed_rows(ids, W + E, 0.5) - O.embed_rows(ids, W - E, 0.5))) / 2e-3
            assert abs(d - g[v, j]) < 1e-9


def test_sample_walks_the_probabilities():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    # order 1, 3, 2, 0 with borders 0.4, 0.7, 0.9, 1
    for u, want in [(0.0, 1), (0.39, 1), (0.41, 3), (0.69, 3), (0.71, 2), (0.89, 2), (0.91, 0), (0.999, 0)]:
        assert O.sample_row(x, u)[0] == want
    i, lp = O.sample_row(x, 0.95, top_k=2)  # 0.4 and 0.3: border 4/7
    assert i == 3 and np.isclose(lp, np.log(3 / 7))
    assert O.sample_row(x, 0.99, top_p=0.39)[0] == 1      # the first alone reaches it
    assert O.sample_row(x, 0.99, top_p=0.41)[0] == 3
    assert O.sample_row(x, 0.99, min_p=0.7)[0] == 3       # 0.4 and 0.3
    assert O.sample_row(x, 0.99, min_p=0.76)[0] == 1
    assert O.sample_row(x, 0.99, top_k=2, top_p=0.5)[0] == 1  # half of 0.7 is reached by 0.4
    assert O.sample_row(x, 0.99, temperature=0)[0] == 1


def test_sample_frequencies_are_the_probabilities():
    rng = np.random.default_rng(2)
    x = rng.standard_normal(6)
    us = (np.arange(20000) + 0.5) / 20000
    got = np.bincount([O.sample_row(x, u, temperature=0.7)[0] for u in us], minlength=6) / 20000
    p = np.exp(x / 0.7)
    assert np.max(np.abs(got - p / p.sum())) < 2e-4  # one cell of the grid per border


@pytest.mark.parametrize("x,u,want", [
    ([-np.inf, np.nan, -np.inf], 0.5, -1),
    ([0.0, np.inf, 1.0, np.inf], 0.6, 3),
    ([1.0, 1.0, 1.0, 1.0], 0.5, 2),
    ([-0.0, 0.0], 0.2, 0),
    ([-np.inf, 2.0], 0.999, 1),
])
def test_sample_edges(x, u, want):
    assert O.sample_row(np.array(x), u)[0] == want


def test_e4m3_values_and_rounding():
    v = O.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[56] == 1.0 and v[-1] == 448.0
    assert np.all(np.diff(v) > 0)
    np.testing.assert_array_equal(O.e4m3_codes(v), np.arange(127))
    np.testing.assert_array_equal(O.e4m3_codes(-v[1:]), np.arange(1, 127) | 128)
    # halfway to the even code, a hair beyond to the nearer one
    assert O.e4m3_codes(np.array([1.0625, 1.1875, 1.0625 + 1e-9, 1.1875 - 1e-9])).tolist() == [56, 58, 57, 57]
    assert O.e4m3_codes(np.array([2.0 ** -10, 3 * 2.0 ** -10, 448.00003, np.nan])).tolist() == [0, 2, 126, 127]


def test_e4m3_against_torch():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * np.float32(60)
    x = np.clip(np.concatenate([x, x * np.float32(1e-4)]), -448, 448)
    np.testing.assert_array_equal(torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), O.e4m3_codes(x))


def test_quantize_round_trip():
    # each value comes back within half a step of its block's scale: 2^-4 of it, or 2^-10 scales
    x = np.random.default_rng(1).standard_normal((200, 300)).astype(np.float32)
    x[7] = 0
    for rows in (1, 128):
        codes, scales = O.quantize(x, rows)
        back = O.dequantize(codes, scales, rows)
        s = np.repeat(np.repeat((scales.T if rows == 1 else scales), rows, 0)[:200], 128, 1)[:, :300]
        assert np.all(np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-6))
        assert np.max(np.abs(back)) >= 0.999 * np.max(np.abs(x))
