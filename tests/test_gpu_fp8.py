"""The 8-bit head on the GPU: quantisers and product against the oracle.

Tolerances.  The quantisers' codes and scales are exact functions of the input:
bit for bit.  A product element is a sum of d terms (exact in fp32: two 4-bit
significands), scaled block sums among them: at most 128 sums within a block,
one sum and two roundings of scales per block.  Counting each as off by a whole
2^-23 (a matrix core may truncate), the error is at most
(128 + blocks + 3) 2^-23 of the sum of magnitudes, and half a step of the output.
bf16 results (but for up to 16 rows under a weight of fewer than 16,384, and one
or two under one of more than 2^28 values, which take the other way) come from the 8-bit matrix instruction, which
aligns the products of 8 k to the largest one's exponent and drops what is 2^-13
of it and less: each of the 7 others loses less than 2^-13 of the largest, so a
group loses at most 7 x 2^-13 of it, and a sum at most 7 x 2^-13 of its magnitudes.
"""
import sys

import numpy as np
import pytest

from oracle import topk_rows
from oracle import vocab_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


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


def randn(shape, seed, dtype="f32", spread=1.0):
    """Normal values whose columns differ in size."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[1]))
    return torch.from_numpy(x.astype(np.float32)).to("cuda:0").to(DT[dtype])


def codes(q):
    return q.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("R,C", [(1, 16), (1, 2880), (3, 128), (130, 144), (257, 400), (128, 256), (1000, 64)])
def test_quantisers_are_exact(ckl, dtype, block_rows, R, C):
    say(f"[case] quantize {dtype} {block_rows} {R}x{C}")
    x = randn((R, C), R + C, dtype)
    x[R // 2] = 0
    x[0, 0] = 1e-42 if dtype == "f32" else 1e-38
    q, s = ckl.quantize_fp8(x, block_rows)
    oc, os_ = O.quantize(x.float().cpu().numpy(), block_rows)
    np.testing.assert_array_equal(s.cpu().numpy(), os_)
    np.testing.assert_array_equal(codes(q), oc)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantiser_edges(ckl, block_rows):
    x = torch.zeros(256, 256, device="cuda:0")
    x[0, :128] = 1e-44                      # a scale below the smallest normal number
    x[1, 5], x[1, 6], x[1, 7] = float("inf"), float("nan"), 3.0
    x[2] = float("-inf")
    x[3, 130] = torch.finfo(torch.float32).max
    x[130:, :128] = torch.linspace(-448, 448, 126 * 128, device="cuda:0").view(126, 128)
    x[200, 128:] = -0.0
    q, s = ckl.quantize_fp8(x, block_rows)
    oc, os_ = O.quantize(x.cpu().numpy(), block_rows)
    np.testing.assert_array_equal(s.cpu().numpy(), os_)
    got = codes(q)
    nan = ~np.isfinite(x.cpu().numpy())
    assert np.all((got[nan] & 127) == 127)
    np.testing.assert_array_equal(got[~nan], oc[~nan])


def test_every_rounding_of_the_type(ckl):
    # all values, midpoints between them and their neighbours, at scale 1
    v = O.e4m3_values()
    mid = (v[1:] + v[:-1]) / 2
    pts = np.concatenate([v, mid, np.nextafter(mid.astype(np.float32), np.float32(0)), np.nextafter(mid.astype(np.float32), np.float32(1e9))])
    pts = np.concatenate([pts, -pts]).astype(np.float32)
    rows = np.zeros((-(-pts.size // 127), 128), np.float32)
    rows[:, 0] = 448.0
    flat = rows[:, 1:].reshape(-1)
    flat[: pts.size] = pts
    rows[:, 1:] = flat.reshape(rows.shape[0], 127)
    q, s = ckl.quantize_fp8(torch.from_numpy(rows).to("cuda:0"))
    assert torch.all(s == 1)
    np.testing.assert_array_equal(codes(q), O.e4m3_codes(rows))


def check_product(ckl, M, V, d, dtype, seed=0, spread=1.0):
    say(f"[case] matmul_fp8 M={M} V={V} d={d} {dtype}")
    xq, xs = ckl.quantize_fp8(randn((M, d), seed + 1, "bf16", spread))
    wq, ws = ckl.quantize_fp8(randn((V, d), seed + 2, "f32", spread) * 0.02, 128)
    out = ckl.matmul_fp8(xq, xs, wq, ws, dtype=DT[dtype])
    x = torch.from_numpy(O.dequantize(codes(xq), xs.cpu().numpy(), 1)).to("cuda:0")
    w = torch.from_numpy(O.dequantize(codes(wq), ws.cpu().numpy(), 128)).to("cuda:0")
    want, mag = x @ w.t(), x.abs() @ w.abs().t()
    lost = 7 * 2.0 ** -13 if dtype == "bf16" and (M > 16 or V >= 16384 and not (M <= 2 and V * d > 1 << 28)) else 0.0
    bound = ((128 + -(-d // 128) + 3) * 2.0 ** -23 + lost) * mag + want.abs() * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)
    err = (out.double() - want).abs()
    assert out.dtype == DT[dtype] and torch.all(err <= bound), float((err - bound).max())
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 64, 65, 200])
@pytest.mark.parametrize("V,d", [(1, 16), (33, 128), (129, 144), (515, 2880), (1000, 1040)])
def test_product_small(ckl, dtype, M, V, d):
    check_product(ckl, M, V, d, dtype, seed=M + V)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,V,d", [(70, 33000, 272), (130, 33001, 272), (300, 40000, 144), (257, 32003, 528), (2000, 5000, 2064),
                                   (129, 66000, 64), (1030, 8200, 128), (16, 50001, 2880), (5, 201088, 2880), (2, 100003, 2880)])
def test_product_of_every_tile_size(ckl, dtype, M, V, d):
    check_product(ckl, M, V, d, dtype, seed=M)


def test_product_is_the_same_for_a_row_alone(ckl):
    # a row's sums do not depend on the rows beside it within one kernel, and
    # every kernel adds blocks of k in an order that stays within the bound
    out = check_product(ckl, 300, 3000, 400, "f32")
    again = check_product(ckl, 300, 3000, 400, "f32")
    assert torch.equal(out, again)


def test_nan_stays_in_its_row_and_column(ckl):
    for M in (4, 100):
        x, w = randn((M, 272), 1), randn((700, 272), 2)
        x[2, 270], w[300, 1] = float("nan"), float("inf")
        out = ckl.logits_fp8(x, *ckl.quantize_fp8(w, 128), dtype=torch.float32)
        bad = torch.isnan(out)
        assert bad[2].all() and bad[:, 300].all() and bad.sum().item() == 700 + M - 1


def test_outputs_of_any_alignment(ckl):
    xq, xs = ckl.quantize_fp8(randn((90, 128), 1))
    wq, ws = ckl.quantize_fp8(randn((640, 128), 2), 128)
    for dtype in DT.values():
        want = ckl.matmul_fp8(xq, xs, wq, ws, dtype=dtype)
        buf = torch.full((90 * 640 + 9,), 7.0, dtype=dtype, device="cuda:0")
        out = buf[1:90 * 640 + 1].view(90, 640)
        assert ckl.matmul_fp8(xq, xs, wq, ws, out=out) is out
        assert torch.equal(out, want) and buf[0] == 7 and torch.all(buf[90 * 640 + 1:] == 7)


def test_offsets_beyond_32_bits(ckl):
    # an output of more than 2^31 elements and a weight of more than 2^31 bytes
    M, V, d = 11000, 201088, 16
    say("[case] matmul_fp8 beyond 2^31 outputs")
    x, w = randn((M, d), 1, spread=0.0), randn((V, d), 2, spread=0.0)
    out = ckl.logits_fp8(x, *ckl.quantize_fp8(w, 128))
    tail = ckl.logits_fp8(x[-200:].contiguous(), *ckl.quantize_fp8(w, 128))
    assert torch.equal(out[-200:], tail)
    del out
    say("[case] matmul_fp8 beyond 2^31 bytes of weight")
    V, d = 800000, 2880
    wq = torch.zeros(V, d, dtype=torch.uint8, device="cuda:0")
    wq[-300:] = 0x38  # 1.0
    ws = torch.ones(V // 128, -(-d // 128), device="cuda:0")
    for M in (2, 70):
        xq, xs = torch.full((M, d), 0x38, dtype=torch.uint8, device="cuda:0").view(torch.float8_e4m3fn), torch.ones(-(-d // 128), M, device="cuda:0")
        out = ckl.matmul_fp8(xq, xs, wq.view(torch.float8_e4m3fn), ws, dtype=torch.float32)
        assert torch.all(out[:, -300:] == d) and not out[:, :-300].any()


def test_logits_to_tokens(ckl):
    # the run of them: rows of an embedding as hidden states, logits under the
    # 8-bit head, sampled tokens, and the lookup of those
    W = randn((3000, 256), 5, "bf16", 0.3)
    wq, ws = ckl.quantize_fp8(W, 128)
    tok = torch.randint(0, 3000, (40,), dtype=torch.int32, device="cuda:0")
    for step in range(3):
        H = ckl.embed(tok, W, 0.5)
        logits = ckl.logits_fp8(H, wq, ws)
        u = torch.rand(40, device="cuda:0")
        tok, logp = ckl.sample(logits, u, temperature=0.8, top_k=50, top_p=0.95)
        host, hu = logits.float().cpu().numpy(), u.cpu().numpy()
        want = [O.sample_row(host[r], hu[r], temperature=0.8, top_k=50, top_p=0.95)[0] for r in range(40)]
        assert tok.tolist() == want and torch.all(logp <= 0)


@pytest.mark.parametrize("chunk", [0, 1, 64, 100])
def test_teacher_topk(ckl, chunk):
    H, W = randn((130, 144), 6, "bf16"), randn((2001, 144), 7, "bf16")
    wq, ws = ckl.quantize_fp8(W, 128)
    ids, vals = ckl.teacher_topk(H, wq, ws, 20, chunk=chunk)
    parts = [ckl.logits_fp8(H[r:r + (chunk or 130)], wq, ws) for r in range(0, 130, chunk or 130)]
    oi, ov = topk_rows(torch.cat(parts).float().cpu().numpy(), 20)
    np.testing.assert_array_equal(ids.cpu().numpy(), oi)
    np.testing.assert_array_equal(vals.cpu().numpy(), ov)


def test_no_rows(ckl):
    wq, ws = ckl.quantize_fp8(randn((300, 64), 1), 128)
    H = torch.empty(0, 64, device="cuda:0")
    assert ckl.logits_fp8(H, wq, ws).shape == (0, 300)
    ids, vals = ckl.teacher_topk(H, wq, ws, 5)
    assert ids.shape == (0, 5) and vals.shape == (0, 5)


def test_two_streams_and_a_graph(ckl):
    x, w = randn((100, 528), 1), randn((4000, 528), 2)
    wq, ws = ckl.quantize_fp8(w, 128)
    want = ckl.logits_fp8(x, wq, ws)
    few = ckl.logits_fp8(x[:3], wq, ws)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(6):
        with torch.cuda.stream(streams[turn % 2]):
            got.append((ckl.logits_fp8(x, wq, ws), ckl.logits_fp8(x[:3], wq, ws)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want) and torch.equal(b, few)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = ckl.logits_fp8(x, wq, ws), ckl.logits_fp8(x[:3], wq, ws)
    for turn in range(3):
        x.mul_(1.3)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, ckl.logits_fp8(x, wq, ws)) and torch.equal(b, ckl.logits_fp8(x[:3], wq, ws))


def test_refusals(ckl):
    from chunked_kl_loss_seq_amd import CklError

    x, w = randn((8, 64), 1), randn((200, 64), 2)
    xq, xs = ckl.quantize_fp8(x)
    wq, ws = ckl.quantize_fp8(w, 128)
    for bad in (lambda: ckl.quantize_fp8(x.half()), lambda: ckl.quantize_fp8(x.cpu()), lambda: ckl.quantize_fp8(x.t()),
                lambda: ckl.quantize_fp8(x, 64), lambda: ckl.matmul_fp8(xq, xs.t().contiguous(), wq, ws),
                lambda: ckl.matmul_fp8(xq, xs, wq[:, :32].contiguous(), ws), lambda: ckl.matmul_fp8(x, xs, wq, ws),
                lambda: ckl.matmul_fp8(xq, xs, wq, ws[:1]), lambda: ckl.matmul_fp8(xq, xs, wq, ws, dtype=torch.float16),
                lambda: ckl.matmul_fp8(xq, xs, wq, ws, out=torch.zeros(8, 199, device="cuda:0")),
                lambda: ckl.logits_fp8(x[0], wq, ws), lambda: ckl.teacher_topk(x, wq, ws, 0),
                lambda: ckl.teacher_topk(x, wq, ws, 201), lambda: ckl.teacher_topk(x, wq, ws, 5, chunk=-1)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(CklError):  # C % 16
        ckl.quantize_fp8(randn((8, 72), 1))
    with pytest.raises(CklError):  # misaligned rows
        ckl.quantize_fp8(torch.zeros(129, device="cuda:0")[1:].view(1, 128))
