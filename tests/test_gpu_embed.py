"""Token embedding and its gradient on the GPU against the float64 oracle.

Tolerances.  The lookup is one fp32 product rounded once to the output type: it
is compared bit for bit with that product and rounding.  A gradient element is
an fp32 sum of n terms in some order, one product with the scale and, when it
is added to dW, one more sum: off by at most (n + 2) 2^-24 times the sum of the
magnitudes (n - 1 sums, the product, the last sum, to first order, and one
more for the terms of second order).
"""
import sys

import numpy as np
import pytest

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


def tokens(rng, N, V, kind):
    if kind == "one":
        return np.full(N, V // 2, np.int32)
    if kind == "none":
        return np.where(np.arange(N) % 2 == 0, -1, V + 5).astype(np.int32)
    if kind == "uniform":
        return rng.integers(0, V, N).astype(np.int32)
    # text: skewed, with padding and ids just outside the vocabulary
    ids = np.minimum((rng.pareto(0.7, N)).astype(np.int64), V - 1).astype(np.int32)
    ids[rng.random(N) < 0.1] = -1
    ids[rng.random(N) < 0.02] = V
    ids[rng.random(N) < 0.02] = np.iinfo(np.int32).min
    return ids


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0")
    return t.to(DT[dtype]) if dtype else t


def check_grad(got, ids, dY, V, scale, base=None):
    want, mag, count = O.embed_grad(ids, dY, V, scale)
    if base is not None:
        want, mag = want + base, mag + np.abs(base)
    err = np.abs(got.astype(np.float64) - want)
    bound = (count[:, None] + 2) * 2.0 ** -24 * mag
    assert np.all(err <= bound), float(np.max(err - bound))
    if base is not None:  # rows of absent tokens as they were
        np.testing.assert_array_equal(got[count == 0], base.astype(np.float32)[count == 0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d", [(1, 1, 8), (1, 5000, 2880), (3, 7, 24), (65, 33, 72), (257, 1000, 520), (5000, 300, 64)])
def test_lookup_is_exact(ckl, dtype, N, V, d):
    say(f"[case] embed {dtype} N={N} V={V} d={d}")
    rng = np.random.default_rng(N + d)
    W = dev(rng.standard_normal((V, d)).astype(np.float32), dtype)
    ids = tokens(rng, N, V, "text")
    for scale in (1.0, 53.66563, -0.3):
        got = ckl.embed(dev(ids), W, scale)
        there = dev((ids >= 0) & (ids < V))
        want = (W.float() * scale).to(DT[dtype])[dev(ids).long().clamp(0, V - 1)]
        want = torch.where(there[:, None], want, torch.zeros_like(want))
        assert got.dtype == DT[dtype] and torch.equal(got.view(torch.uint8), want.contiguous().view(torch.uint8))


def test_lookup_shapes_and_out(ckl):
    W = torch.randn(50, 16, device="cuda:0")
    ids = torch.randint(0, 50, (3, 4, 5), dtype=torch.int32, device="cuda:0")
    out = torch.empty(3, 4, 5, 16, device="cuda:0")
    got = ckl.embed(ids, W, out=out)
    assert got is out and torch.equal(got, W[ids.long()])
    assert torch.equal(ckl.embed(ids[1, 2, 3], W), W[ids[1, 2, 3].long()])
    assert ckl.embed(ids[:0], W).shape == (0, 4, 5, 16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["text", "uniform", "one", "none"])
@pytest.mark.parametrize("N,V,d", [(1, 3, 8), (15, 40, 64), (16, 64, 520), (17, 31, 24), (300, 65, 72), (4099, 500, 40),
                                   (8192, 100, 16), (8193, 3000, 32)])
def test_gradient(ckl, dtype, kind, N, V, d):
    # tiles of 16 and 32 positions, both sorts, runs inside a tile, across two
    # and across all of them, columns that end inside a slice
    say(f"[case] embed_bwd {dtype} {kind} N={N} V={V} d={d}")
    rng = np.random.default_rng(7 * N + d)
    ids = tokens(rng, N, V, kind)
    dY = dev(rng.standard_normal((N, d)).astype(np.float32), dtype)
    host = dY.float().cpu().numpy()
    got = ckl.embed_bwd(dev(ids), dY, V, 1.7)
    check_grad(got.cpu().numpy(), ids, host, V, 1.7)
    base = rng.standard_normal((V, d)).astype(np.float32)
    acc = dev(base)
    assert ckl.embed_bwd(dev(ids), dY, V, 1.7, dW=acc, accumulate=True) is acc
    check_grad(acc.cpu().numpy(), ids, host, V, 1.7, base.astype(np.float64))
    # a fixed order: the same bits again, over memory that held something else
    again = ckl.embed_bwd(dev(ids), dY, V, 1.7, dW=torch.full((V, d), float("nan"), device="cuda:0"))
    assert torch.equal(again, got)


@pytest.mark.parametrize("kind", ["text", "uniform", "one", "none"])
@pytest.mark.parametrize("N,V,d", [(63, 64, 520), (64, 10, 8), (65, 1000, 24), (255, 33, 1032), (256, 97, 256), (257, 97, 256)])
def test_gradient_of_few_positions(ckl, kind, N, V, d):
    # up to 256 positions take one launch: occurrences in each group of 64
    # positions, more than 16 of them in one, and the first count past it
    test_gradient(ckl, "bf16" if N % 2 else "f32", kind, N, V, d)


@pytest.mark.parametrize("N,V", [(70001, 400000), (20000, 262143), (20000, 262144), (9000, 1 << 20)])
def test_gradient_of_large_vocabularies(ckl, N, V):
    # keys of 18 bits and more: two and three radix passes; 70,001 positions: tiles of 64
    say(f"[case] embed_bwd large vocabulary N={N} V={V}")
    rng = np.random.default_rng(V)
    ids = rng.integers(0, V, N).astype(np.int32)
    ids[: N // 4] = V - 1
    ids[N // 4: N // 3] = 511
    rng.shuffle(ids)
    dY = rng.standard_normal((N, 8)).astype(np.float32)
    got = ckl.embed_bwd(dev(ids), dev(dY), V)
    check_grad(got.cpu().numpy(), ids, dY, V, 1.0)


def test_offsets_beyond_32_bits(ckl):
    # a table and a gradient of more than 2^31 elements
    V, d = 800000, 2880
    say("[case] embed beyond 2^31 elements")
    W = torch.empty(V, d, dtype=torch.bfloat16, device="cuda:0")
    W[-3:] = torch.randn(3, d, device="cuda:0").to(torch.bfloat16)
    ids = torch.tensor([V - 1, V - 3, V - 1], dtype=torch.int32, device="cuda:0")
    out = ckl.embed(ids, W)
    assert torch.equal(out, W[ids.long()])
    del W
    dY = torch.randn(3, d, device="cuda:0")
    dW = ckl.embed_bwd(ids, dY, V)
    assert torch.equal(dW[V - 1], dY[0] + dY[2]) and torch.equal(dW[V - 3], dY[1])
    assert not dW[V - 2].any() and not dW[: V - 3].any()


def test_empty_batch(ckl):
    ids = torch.empty(0, dtype=torch.int32, device="cuda:0")
    dY = torch.empty(0, 16, device="cuda:0")
    assert not ckl.embed_bwd(ids, dY, 9, dW=torch.ones(9, 16, device="cuda:0")).any()
    assert ckl.embed_bwd(ids, dY, 9, dW=torch.ones(9, 16, device="cuda:0"), accumulate=True).all()


def test_non_finite_rows_stay_in_their_token(ckl):
    ids = torch.tensor([1, 2, 1, -1], dtype=torch.int32, device="cuda:0")
    dY = torch.ones(4, 8, device="cuda:0")
    dY[0] = float("inf")
    dY[3] = float("nan")  # a position without a token
    dW = ckl.embed_bwd(ids, dY, 4)
    assert torch.isinf(dW[1]).all() and torch.equal(dW[2], dY[1]) and not dW[0].any() and not dW[3].any()


def test_autograd(ckl):
    rng = np.random.default_rng(3)
    ids = tokens(rng, 200, 50, "text")
    for dtype in ("bf16", "f32"):
        W = dev(rng.standard_normal((50, 24)).astype(np.float32), dtype).requires_grad_()
        g = dev(rng.standard_normal((200, 24)).astype(np.float32), dtype)
        ckl.embedding(dev(ids), W, 3.0).backward(g)
        assert W.grad.dtype == W.dtype
        want = ckl.embed_bwd(dev(ids), g, 50, 3.0)
        assert torch.equal(W.grad, want.to(W.dtype))


def test_tied_weights_add_to_the_head_gradient(ckl):
    # one table for the lookup and the head: the loss writes dW and the
    # lookup's gradient is added to it, as autograd's sum of both
    from chunked_kl_loss_seq_amd import workloads as WL

    inp = WL.small(300, 64, 500, 20, dtype="f32", seed=4)
    W, ids, T = dev(inp["W"]), dev(inp["ids"]), dev(inp["tlogit"])
    text = torch.randint(0, 500, (300,), dtype=torch.int32, device="cuda:0")
    H = ckl.embed(text, W, 8.0)
    loss, dH, dW = ckl.fwd_bwd(H, W, ids, T)
    head = dW.clone()
    ckl.embed_bwd(text, dH, 500, 8.0, dW=dW, accumulate=True)
    Wt = W.clone().requires_grad_()
    ckl.fused_kl(ckl.embedding(text, Wt, 8.0), Wt, ids, T).backward()
    both = head + ckl.embed_bwd(text, dH, 500, 8.0)
    assert torch.allclose(dW, both, rtol=2e-6, atol=1e-9) and torch.allclose(Wt.grad, both, rtol=2e-6, atol=1e-9)
    # and it is the derivative of the loss: a step along a direction E
    E = torch.randn_like(W)

    def difference(s):
        d = []
        for step in (s, -s):
            Ws = (W.double() + step * E.double())
            z = (Ws[text.long()] * 8.0) @ Ws.t()
            p = torch.softmax(T.double(), 1)
            lp = torch.log_softmax(z, 1).gather(1, ids.long())
            d.append(((p * (p.log() - lp)).sum(1)).mean().item())
        return (d[0] - d[1]) / (2 * s)

    # A central difference is off by s^2 f3 / 6 + s^4 f5 / 120 + ..; two of them
    # cancel the first term.  Along E a logit is z0 + a s + b s^2 with a of about 8
    # x sqrt(2 x 64) x 0.02 = 2 and b of about 8 x 8 = 64, so f3 goes as 3 a b and
    # f5 as 15 a b^2: the second term is s^2 / 20 x 5 b = 2e-5 of the first, and a
    # hundredth of the difference between the two steps covers what is left.
    wide, narrow = difference(1e-3), difference(5e-4)
    slope, off = (4 * narrow - wide) / 3, 0.01 * abs(wide - narrow) + 1e-10
    # The gradient's error e has a norm below 1e-5 of each part's (the fp32 path's
    # bound on dW, and on dH, whose rows add up in groups of up to m positions).
    # E is drawn apart from it, so e . E is normal with deviation |e|: six of them.
    m = torch.bincount(text.long()).max().item()
    e = 1e-5 * (head.double().norm() + 8.0 * m ** 0.5 * dH.double().norm()).item()
    assert abs(slope - (dW.double() * E.double()).sum().item()) <= 6 * e + off


def test_two_streams_at_once(ckl):
    rng = np.random.default_rng(5)
    jobs = []
    for i in range(2):
        ids = dev(tokens(rng, 20000, 3000, "text"))
        dY = dev(rng.standard_normal((20000, 256)).astype(np.float32))
        jobs.append((ids, dY, ckl.embed_bwd(ids, dY, 3000)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(5):
        for (ids, dY, _w), s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(ckl.embed_bwd(ids, dY, 3000))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, jobs[i % 2][2])


def test_captured_and_replayed(ckl):
    # two graphs, each with the lookup and its gradient, replayed in turn with
    # eager calls between; every replay against the eager result
    rng = np.random.default_rng(6)
    W = dev(rng.standard_normal((3000, 64)).astype(np.float32))
    parts = []
    for N in (700, 9000):
        ids = dev(tokens(rng, N, 3000, "text"))
        dY = dev(rng.standard_normal((N, 64)).astype(np.float32))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ckl.embed(ids, W), ckl.embed_bwd(ids, dY, 3000)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, dW = ckl.embed(ids, W, 2.0), ckl.embed_bwd(ids, dY, 3000, 2.0)
        parts.append((ids, dY, g, out, dW))
    for turn in range(3):
        for ids, dY, g, out, dW in parts:
            ids.copy_(torch.roll(ids, 11))
            dY.mul_(1.5)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ckl.embed(ids, W, 2.0)) and torch.equal(dW, ckl.embed_bwd(ids, dY, 3000, 2.0))


def test_embedding_under_capture(ckl, monkeypatch):
    # an eager graph of the same leaf may live: a captured call that needs its
    # gradient is refused before anything is recorded; without one it replays
    rng = np.random.default_rng(8)
    ids = dev(tokens(rng, 50, 100, "uniform"))
    W = dev(rng.standard_normal((100, 16)).astype(np.float32)).requires_grad_(True)
    eager = ckl.embedding(ids, W, 2.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with torch.no_grad():
            out = ckl.embedding(ids, W, 2.0)
        with pytest.raises(RuntimeError, match="capture embed and embed_bwd"):
            ckl.embedding(ids, W)
    for _ in range(3):
        ids.copy_(torch.roll(ids, 3))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ckl.embed(ids, W.detach(), 2.0))
    # the backward's own check (reported as capturing, nothing is captured)
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError, match="capture embed and embed_bwd"):
            eager.sum().backward()
    assert W.grad is None
    ckl.embedding(ids, W, 2.0).sum().backward()
    assert torch.equal(W.grad, ckl.embed_bwd(ids, torch.ones(50, 16, device="cuda:0"), 100, 2.0))


def test_refusals(ckl):
    W = torch.zeros(10, 16, device="cuda:0")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    dY = torch.zeros(4, 16, device="cuda:0")
    for bad in (lambda: ckl.embed(ids.long(), W), lambda: ckl.embed(ids, W.half()), lambda: ckl.embed(ids, W.t()),
                lambda: ckl.embed(ids, W.cpu()), lambda: ckl.embed(ids.cpu(), W), lambda: ckl.embed(ids[::2], W),
                lambda: ckl.embed(ids, W, out=torch.zeros(4, 8, device="cuda:0")),
                lambda: ckl.embed_bwd(ids, dY[:3], 10), lambda: ckl.embed_bwd(ids, dY.t().contiguous(), 10),
                lambda: ckl.embed_bwd(ids, dY, 10, accumulate=True),
                lambda: ckl.embed_bwd(ids, dY, 10, dW=torch.zeros(9, 16, device="cuda:0")),
                lambda: ckl.embed_bwd(ids, dY, 10, dW=torch.zeros(10, 16, device="cuda:0", dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            bad()
    from chunked_kl_loss_seq_amd import CklError

    with pytest.raises(CklError):  # d % 8
        ckl.embed(ids, torch.zeros(10, 12, device="cuda:0"))
    with pytest.raises(CklError):
        ckl.embed_bwd(ids, dY, 0)
    with pytest.raises(CklError):  # misaligned rows
        ckl.embed(ids, torch.zeros(161, device="cuda:0")[1:].view(10, 16))
