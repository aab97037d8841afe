"""The residual's norms over more rows than the card holds at once, on the GPU against the float64 oracle: every workgroup
goes over several rows (or several sets of rows side by side), whose values come in while the ones before are worked on.

Tolerances as in test_gpu_residual."""
import pytest

from test_gpu_residual import check, ckl  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_at_once(d):
    """No grid of either direction holds more: 256 compute units of at most 32 waves of 64 lanes, a lane at most two vectors
    of 8 of a row (one where several rows share a wave, which takes lanes in powers of two)."""
    vectors = d // 8
    if vectors > 64:
        return 256 * 32 // -(-vectors // 128)
    lanes = 1
    while lanes < vectors:
        lanes *= 2
    return 256 * 32 * (64 // lanes)


# rows in one lane, in 16 and 64 of them, in a wave by two vectors, in several waves, in more than 512 threads (backward;
# both directions in the last), the last turn a short one
SIZES = [(524609, 8), (33001, 72), (8501, 512), (8501, 520), (4301, 1032), (2801, 2880), (1701, 4104), (1001, 8200)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,p", [("vector", 0.2), ("full", 0.1)])
@pytest.mark.parametrize("N,d", SIZES)
def test_turns(ckl, dtype, gate, p, N, d):  # noqa: F811
    assert N > rows_at_once(d)
    check(ckl, dtype, N, d, True, True, gate, p)


@pytest.mark.parametrize("N,d", [(33001, 72), (2801, 2880)])
def test_turns_without_a_norm_or_dropout(ckl, N, d):  # noqa: F811
    assert N > rows_at_once(d)
    check(ckl, "f32", N, d, False, True, "none", 0.0)
    check(ckl, "bf16", N, d, True, False, "vector", 0.0)
