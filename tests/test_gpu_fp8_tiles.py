"""The 8-bit product at sizes that reach its largest tile, many blocks of k and
rows taken alone, against the definition in 64 bits.

Tolerances.  The sum of the block products is off by at most (128 + blocks + 3)
2^-23 of the sum of the magnitudes (at most 128 sums within a block, one sum and
two roundings of scales a block, each counted as a whole 2^-23 as a matrix core
may truncate), and the result by half a step of its type.  For bf16 results the
8-bit matrix instruction loses less than 7 x 2^-13 of the magnitudes more.
"""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ckl():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for these tests")
    import chunked_kl_loss_seq_amd as m
    from chunked_kl_loss_seq_amd import binding

    binding.lib()
    return m


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def operands(ckl, M, V, d, seed):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    size = torch.randn(d, device="cuda:0", generator=g).exp()  # columns differ in size
    x = (torch.randn(M, d, device="cuda:0", generator=g) * size).to(BF16)
    w = torch.randn(V, d, device="cuda:0", generator=g) * size * 0.02
    return (x, *ckl.quantize_fp8(x), *ckl.quantize_fp8(w, 128))


def check(out, xq, xs, wq, ws, rows=slice(None)):
    """out against the product of the values that codes and scales stand for."""
    d, V = wq.shape[1], wq.shape[0]
    x = xq.double()[rows] * xs.double().t()[rows].repeat_interleave(128, 1)[:, :d]
    blocks = xs.shape[0]
    for v in range(0, V, 16384):
        s = ws[v // 128:v // 128 + 128].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        w = wq[v:v + 16384].double()
        w = w * s[:w.shape[0], :d]
        want, mag = x @ w.t(), x.abs() @ w.abs().t()
        lost = 7 * 2.0 ** -13 if out.dtype == BF16 else 0.0
        half_step = 2.0 ** -8 if out.dtype == BF16 else 2.0 ** -24
        bound = ((128 + blocks + 3) * 2.0 ** -23 + lost) * mag + want.abs() * half_step
        err = (out[:, v:v + 16384].double() - want).abs()
        assert torch.all(err <= bound), (v, float((err - bound).max()))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,V,d", [
    (2048, 40000, 400),   # 256 x 256 tiles, whole rows of 16 bytes, four blocks of k, the last of 16
    (1999, 40001, 272),   # the same with ragged ends in rows, ids and k, rows of any alignment
    (2048, 40000, 128),   # one whole block
    (1030, 66003, 2880),  # 128 x 128 tiles
])
def test_large_tiles(ckl, dtype, M, V, d):
    say(f"[case] matmul_fp8 M={M} V={V} d={d} {dtype}")
    _, xq, xs, wq, ws = operands(ckl, M, V, d, M + d)
    out = ckl.matmul_fp8(xq, xs, wq, ws, dtype=dtype)
    assert out.dtype == dtype
    check(out, xq, xs, wq, ws)
    assert torch.equal(out, ckl.matmul_fp8(xq, xs, wq, ws, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,V", [(2049, 32769), (260, 17000), (130, 17000), (65, 9000), (5, 3000)])
@pytest.mark.parametrize("d", [8192, 8336, 16400])
def test_more_blocks_than_lanes(ckl, dtype, M, V, d):
    # a wave holds the weight scales of 64 blocks of k, one a lane: 64, 66 and
    # 129 blocks, for every tile (256 x 256 .. 64 x 64) and the few-row kernel
    if M > 2000 and d > 10000:
        d = 12304  # 97 blocks; keeps the reference's time down
    say(f"[case] matmul_fp8 M={M} V={V} d={d} {dtype}")
    _, xq, xs, wq, ws = operands(ckl, M, V, d, M + d)
    out = ckl.matmul_fp8(xq, xs, wq, ws, dtype=dtype)
    check(out, xq, xs, wq, ws)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_alone(ckl, dtype):
    # every tile adds a row's blocks of k in one order, so a row's results are
    # the same bits under any tile, whatever the rows beside it (32,769 ids: tiles
    # for any number of rows)
    say(f"[case] rows alone {dtype}")
    x, xq, xs, wq, ws = operands(ckl, 2049, 32769, 528, 5)
    out = ckl.matmul_fp8(xq, xs, wq, ws, dtype=dtype)
    for r, n in ((0, 300), (1900, 149), (1024, 70), (7, 17), (2040, 9), (2048, 1), (300, 2)):
        assert torch.equal(ckl.logits_fp8(x[r:r + n], wq, ws, dtype=dtype), out[r:r + n]), (r, n)
    # up to 16 rows under fewer than 16,384 ids: another kernel, within the bound
    few = ckl.matmul_fp8(xq[:9].contiguous(), xs[:, :9].contiguous(), wq[:9000].contiguous(), ws[:71].contiguous(),
                         dtype=dtype)
    check(few, xq, xs, wq[:9000], ws[:71], slice(0, 9))
