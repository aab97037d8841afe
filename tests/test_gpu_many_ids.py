"""dH of vocabularies so large that a tile of 256 rows of the gradient passes 2 GiB, on the GPU: every row, against
float64 on the same device.

Tolerance of a row of dH = G W, with h = 2^-24, e half a step of the path's type and a = sum |G| |W|:
  G     held in the path's type, e; p = exp(z - lse) within 5e-3 of its value: a logit is an fp32 sum of d products, off by
        at most (d + 8) h sum |H| |W| (1e-3 here at d = 2,048 but for the given ids, whose p is below 1e-2 with 1.2e-2), twice
        for the lse's, whose sums of at most 400 terms in a chain add 400 h.
  sum   over the ids in `runs` runs and then those: (V / runs + 32) h a.  The runs are what the library takes for these
        sizes: 31 for the loss, 16 and 12 for the hidden states.
  half a step of the output.
The two given ids of a row make most of it, so that a row that is read as zeros is off by more than ten times that."""
import sys

import pytest

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


def expect(H, W, rows, put):
    """(dH, sum |G| |W|) of the rows in float64, G = (put - sum put x softmax) by blocks of ids; put: row -> {id: weight}."""
    h = H[rows].double()
    V, step = W.shape[0], 1 << 19
    parts = [torch.logsumexp(h @ W[v:v + step].double().t(), 1) for v in range(0, V, step)]
    lse = torch.logsumexp(torch.stack(parts), 0)
    total = torch.tensor([sum(put[r].values()) for r in rows], dtype=torch.float64, device=H.device)
    dH, mag = torch.zeros_like(h), torch.zeros_like(h)
    for v in range(0, V, step):
        w = W[v:v + step].double()
        G = -torch.exp(h @ w.t() - lse[:, None]) * total[:, None]
        for i, r in enumerate(rows):
            for j, x in put[r].items():
                if v <= j < v + step:
                    G[i, j - v] += x
        dH += G @ w
        mag += G.abs() @ w.abs()
    return dH, mag


def agree(got, want, mag, dtype, chain, what):
    e = torch.finfo(DT[dtype]).eps / 2
    bound = (e + 5e-3 + (chain + 32) * 2.0 ** -24) * mag
    bound += e * (want.abs() + bound)
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), (what, float((err / bound).max()))
    assert bool((want.abs().amax(1) > 10 * bound.amax(1)).all())  # rows of zeros would not pass


def weights(g, V, d, dtype):
    W = torch.empty(V, d, device="cuda:0", dtype=DT[dtype])
    return W.normal_(std=0.3, generator=g)


@pytest.fixture(autouse=True)
def room(monkeypatch):
    monkeypatch.setenv("CKL_WORKSPACE_BYTES", str(24 << 30))  # the loss's copy of W has 64 columns at least


# both sides of the tiles of 256 rows, and beyond those of 128
@pytest.mark.parametrize("dtype,N,V", [("bf16", 256, 5592000), ("bf16", 256, 6000000), ("bf16", 130, 16900000),
                                       ("f32", 256, 2796000), ("f32", 256, 2900000), ("f32", 70, 8500000)])
def test_loss(ckl, dtype, N, V):
    say(f"[case] loss {dtype} N={N} V={V}")
    d, K = 8, 2
    g = torch.Generator(device="cuda:0")
    g.manual_seed(V)
    H = (torch.randn(N, d, device="cuda:0", generator=g) * 0.2).to(DT[dtype])
    W = weights(g, V, d, dtype)
    first = torch.arange(N, device="cuda:0") * (V // N)
    ids = torch.stack([first, first + V // (2 * N)], 1).to(torch.int32)
    W[ids[:, 0].long()] = torch.ones(d, device="cuda:0", dtype=DT[dtype]) * 2
    W[ids[:, 1].long()] = torch.ones(d, device="cuda:0", dtype=DT[dtype]) * 3
    _, dH, _ = ckl.fwd_bwd(H, W, ids, torch.zeros(N, K, device="cuda:0"))
    rows = sorted({0, 63, 64, N // 2, 127 % N, 128 % N, 191 % N, 192 % N, N - 1})
    put = {r: {int(i): -0.5 / N for i in ids[r]} for r in rows}
    want, mag = expect(H, W, rows, put)
    agree(dH[rows], want, mag, dtype, V / 31, "dH")
    loss, lse = ckl.fwd(H, W, ids, torch.zeros(N, K, device="cuda:0"))
    one = torch.ones((), device="cuda:0")
    dH2, _ = ckl.bwd(H, W, ids, torch.zeros(N, K, device="cuda:0"), lse, grad_loss=one)
    agree(dH2[rows], want, mag, dtype, V / 31, "dH of the recomputing call")


# a width at which tiles of 256 (bf16) and 128 rows (fp32) would be the fastest
@pytest.mark.parametrize("dtype,N,V,d,runs", [("bf16", 200, 5600000, 2048, 16), ("f32", 70, 8400000, 2048, 12)])
def test_hidden_states(ckl, dtype, N, V, d, runs):
    say(f"[case] head {dtype} N={N} V={V} d={d}")
    g = torch.Generator(device="cuda:0")
    g.manual_seed(V)
    H = (torch.randn(N, d, device="cuda:0", generator=g) * 0.02).to(DT[dtype])
    W = weights(g, V, d, dtype)
    first = torch.arange(N, device="cuda:0") * (V // N)
    ids = torch.stack([first, first + V // (2 * N)], 1).to(torch.int32)
    W[ids[:, 0].long()] = torch.ones(d, device="cuda:0", dtype=DT[dtype]) * 2
    W[ids[:, 1].long()] = torch.ones(d, device="cuda:0", dtype=DT[dtype]) * 3
    out = ckl.head_logprobs(H, W, ids)
    one = torch.ones(N, 2, device="cuda:0")
    dH, dW = ckl.head_logprobs_bwd(H, W, ids, *out, one)
    del dW
    rows = sorted({0, 63, 64, N - 6, 127 % N, 128 % N, 191 % N, 192 % N, N - 1})
    want, mag = expect(H, W, rows, {r: {int(i): 1.0 for i in ids[r]} for r in rows})
    agree(dH[rows], want, mag, dtype, V / runs, "dH")
