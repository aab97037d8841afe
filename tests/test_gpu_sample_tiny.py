"""Sampling from bf16 rows whose logits below 2^-24 matter.

Such logits are counted as 0, so a row in which the difference to 0 shows has to
be seen again: at temperatures so low that 2^-24 / T is not small, where min_p's
border falls between 0 and one of them, and where one of them is the largest.
Tokens have to equal the definition's; a log-probability is rounded once to fp32
from masses good to 1e-11.
"""
import sys

import numpy as np
import pytest

from oracle import vocab_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ckl():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for these tests")
    import chunked_kl_loss_seq_amd as m
    from chunked_kl_loss_seq_amd import binding

    binding.lib()
    return m


def check(ckl, row, us, what, **how):
    """The same row under each of the random numbers, against the definition."""
    print(f"[case] sample {what} V={len(row)} {how}", file=sys.stderr, flush=True)
    x = torch.tensor(row, dtype=torch.float32).bfloat16()
    assert np.array_equal(x.double().numpy(), np.asarray(row, np.float64)), "bf16 holds the row"
    u = torch.tensor(us, dtype=torch.float32)
    ids, logp = ckl.sample(x.to("cuda:0").expand(len(us), len(row)), u.to("cuda:0"), **how)
    got = []
    for r, v in enumerate(u.tolist()):
        i, lp = O.sample_row(x.float().numpy(), v, **how)
        assert ids[r].item() == i, (r, v, ids[r].item(), i)
        assert abs(logp[r].item() - lp) <= 2.0 ** -24 * abs(lp) + 1e-11, (r, logp[r].item(), lp)
        got.append(i)
    return got


US = [0.1, 0.3, 0.5, 0.7, 0.9, 0.99]


@pytest.mark.parametrize("T", [2e-8, 4e-9, 1.5e-9, 1e-9, 1e-10, 1e-12])
@pytest.mark.parametrize("fill", [0, 7, 33000])
def test_low_temperatures(ckl, T, fill):
    # the largest logit at or just above 2^-24, or itself below, and others a
    # step or a few below it; beside them logits that weigh nothing
    tail = [-1.0] * fill
    step = 2.0 ** -32  # of bf16 below 2^-24
    for top in (2.0 ** -24, 2.0 ** -24 * (1 + 2.0 ** -7), 2.0 ** -24 - step, 2.0 ** -23):
        check(ckl, [top] + [2.0 ** -24 - 2 * step] * 3 + tail, US, "tiny beside the largest", temperature=T)
        check(ckl, [0.0, 2.0 ** -24 - 2 * step, -2.0 ** -24 + step, top, -0.0] + tail, US,
              "tiny, zeros and the largest", temperature=T)
        check(ckl, [top] + [2.0 ** -24 - 2 * step] * 3 + tail, US, "tiny beside the largest", temperature=T, top_p=0.6)
    got = check(ckl, [2.0 ** -24] + [2.0 ** -24 - step] * 3 + tail, US, "tiny beside 2^-24", temperature=T)
    if T >= 1e-9:  # each of the three weighs 0.79 and more of the largest
        assert len(set(got)) > 2


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_min_p_between_zero_and_tiny(ckl, sign):
    # 1,024 equal largest logits, 100 tiny ones, and one 0: e differs by 3e-8 of
    # itself between the last two, and min_p lies between them.  The 100 weigh 6e-7
    # of the largest ones together, which moves the border that u is next to.
    row = [12.0] * 1024 + [sign * 2.0 ** -25] * 100 + [0.0]
    min_p = float(np.exp(-12.0) * (1 + sign * 1.5e-8))
    us = [np.float32(k / 1024) * np.float32(1 - 2.0 ** -24) for k in range(513, 1024, 17)]
    check(ckl, row, us, "min_p beside 0", min_p=min_p)
    check(ckl, row, us, "min_p beside 0", min_p=min_p, top_k=1100)


@pytest.mark.parametrize("V", [5001, 40001, (1 << 20) + 1])
@pytest.mark.parametrize("top,edge", [(2.0 ** -25, -1.5e-8), (-2.0 ** -25, 1.5e-8)])
def test_largest_is_tiny(ckl, V, top, edge):
    # every e is relative to the largest logit, so min_p's border follows it:
    # below it the largest alone is kept, above it everything
    row = np.full(V, -2.0 ** -7)
    row[V // 2] = top
    got = check(ckl, row, [0.3, 0.8], "largest is tiny", min_p=float(np.exp(-2.0 ** -7) * (1 + edge)))
    assert (set(got) == {V // 2}) == (top > 0)
