"""Sampling from rows that hold NaN of every kind: quiet and signalling ones of
either sign, at the ends of a row, around its largest logit and everywhere.
Such tokens are never drawn, so a row gives what it gives with -inf in their
places, bit for bit."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

KINDS = {torch.bfloat16: (torch.int16, [0x7F81, -0x7F, 0x7FC0, -0x40, 0x7FBF]),
         torch.float32: (torch.int32, [0x7F800001, -0x7FFFFF, 0x7FC00000, -0x400000, 0x7FBFFFFF])}
HOW = [{}, {"temperature": 0.0}, {"top_k": 5}, {"top_k": 700}, {"top_p": 0.5}, {"min_p": 0.05}, {"temperature": 8.0}]


@pytest.fixture(scope="module")
def ckl():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for these tests")
    import chunked_kl_loss_seq_amd as m
    from chunked_kl_loss_seq_amd import binding

    binding.lib()
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V", [(9, 1), (9, 7), (9, 100), (9, 5003), (3, 40001), (70, 9000)])
def test_nan_is_never_drawn(ckl, dtype, N, V):
    as_int, kinds = KINDS[dtype]
    g = torch.Generator().manual_seed(V)
    x = (3 * torch.randn(N, V, generator=g)).to(dtype)
    u = torch.rand(N, generator=g).to("cuda:0")
    for k, bits in enumerate(kinds):
        nan = torch.rand(N, V, generator=g) < (0.1, 0.5, 0.9)[k % 3]
        nan[0] = True  # nothing else
        if N > 3:
            top = x[1:4].float().argmax(1)
            for r, t in enumerate(top.tolist()):  # beside the largest, which stays
                nan[1 + r, max(0, t - 9):t + 9] = True
                nan[1 + r, t] = False
            nan[4, 1:] = False  # the first, the last
            nan[5, :-1] = False
        y = x.clone()
        y[nan] = -float("inf")
        z = x.clone().view(as_int)
        z[nan] = bits
        z, y = z.view(dtype).to("cuda:0"), y.to("cuda:0")
        for how in HOW:
            print(f"[case] sample NaN {bits & 0xFFFFFFFF:08x} N={N} V={V} {dtype} {how}", file=sys.stderr, flush=True)
            got, want = ckl.sample(z, u, **how), ckl.sample(y, u, **how)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert got[0][0].item() == -1 and not nan[torch.arange(N), got[0].cpu().long()][got[0].cpu() >= 0].any()
