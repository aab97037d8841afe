"""The teacher cache past the default chunk: its values are those of one call of
the product on all rows, bit for bit."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_last_chunk_is_no_few_row_call():
    # 33,550 rows under 16,000 ids pass the default chunk by 14 rows, which alone
    # would go by the few-row kernel, whose products are summed without loss
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for these tests")
    import chunked_kl_loss_seq_amd as ckl

    print("[case] teacher_topk past the default chunk", file=sys.stderr, flush=True)
    N, V, d, K = 33550, 16000, 400, 1000
    g = torch.Generator(device="cuda:0")
    g.manual_seed(9)
    H = torch.randn(N, d, device="cuda:0", generator=g).to(torch.bfloat16)
    wq, ws = ckl.quantize_fp8(torch.randn(V, d, device="cuda:0", generator=g) * 0.02, 128)
    ids, vals = ckl.teacher_topk(H, wq, ws, K)
    want = ckl.topk(ckl.logits_fp8(H, wq, ws), K)
    assert torch.equal(ids, want[0]) and torch.equal(vals, want[1])
