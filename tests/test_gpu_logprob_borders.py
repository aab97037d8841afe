"""Alternatives at the numbers and lengths where their bound is taken in another way, on the GPU: up to 24 it comes from the
maxima of 64 groups of threads, above from the threads' own; rows of up to 1,024 go to one wave, of up to 8,192 to 256
threads, longer ones and more than 128 alternatives to 512; few long rows are cut in slices.

Ids exact, tolerances of the rest as in test_gpu_logprob."""
import numpy as np
import pytest

from test_gpu_logprob import check, ckl, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [23, 24, 25, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("kind", ["bulk", "few values", "rising"])
def test_borders(ckl, dtype, top, kind):  # noqa: F811
    rng = np.random.default_rng(top)
    for N, V in ((3, 1023), (3, 1025), (3, 4099), (3, 8191), (256, 8193), (2, 8192), (2, 16390), (300, 10007)):
        check(ckl, make(rng, N, V, kind), dtype, 0, top, rng, grad=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [1, 24, 25, 128, 400])
@pytest.mark.parametrize("at", [300.0, -5000.0])
def test_a_common_offset(ckl, dtype, top, at):  # noqa: F811
    """Logits that share their leading bits by the thousand: the bound's 16 do not tell them apart, a search does."""
    rng = np.random.default_rng(top)
    for N, V in ((2, 700), (2, 6000), (2, 40001), (256, 9001)):
        check(ckl, make(rng, N, V, "bulk") + at, dtype, 0, top, rng, grad=False)
