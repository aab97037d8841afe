"""How near a border may lie: a top-p border off a token's edge by the stated
1e-13 + V / 2^62 of the total falls on the right side of it.

A row holds one largest logit and V - 1 equal ones, each of mass e, so that the
first r tokens weigh 1 + (r - 1) e.  top_p is put just below and just above that
share of the total; u next to 1 then draws the last token kept, whose id is its
place.  The equal logits round alike, which is the worst that the sums can meet."""
import sys

import numpy as np
import pytest

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [3001, 100003, 1 << 20, 1 << 22])
def test_top_p_beside_an_edge(ckl, dtype, V):
    u = torch.tensor([1 - 2.0 ** -24], device="cuda:0")
    off = 1e-13 + V / 2.0 ** 62
    for drop in (0.0078125, 0.3359375, 1.0, 2.71875, 7.15625, 12.125):  # bf16 numbers
        x = torch.full((1, V), -drop, dtype=dtype, device="cuda:0")
        x[0, 0] = 0.25
        e = np.exp(-np.longdouble(drop + 0.25))
        total = 1 + (V - 1) * e
        for r in (V // 3, V // 2, V - 7):
            share = (1 + (r - 1) * e) / total
            for p, keep in ((float(share - off), r), (float(share + off), r + 1)):
                print(f"[case] top-p beside an edge V={V} {dtype} drop={drop} r={r}", file=sys.stderr, flush=True)
                ids, _ = ckl.sample(x, u, top_p=p)
                assert ids.item() == keep - 1, (drop, r, p)
