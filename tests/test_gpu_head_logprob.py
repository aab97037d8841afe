"""Log-probabilities from hidden states on the GPU, and their gradients, against the float64 oracle.

Tolerances beside those of the logits' form (test_gpu_logprob), with h = 2^-24:
  a logit is an fp32 sum of d products in some order: off by tz = (d + 8) h sum |H| |W|; E = the row's largest tz.
  log-normaliser  E more;  logp  tz + E more;  entropy  E sum p |log p + H| more;  l = log p in the gradient  tz + E more.
  G               its own error as in the logits' form, and half a step of the path's type (it is held in it)
  dH, dW          sums of V and N products: (errors of G) |W| and |H|, (terms + 16) h sum |G| |W| (and |H|), half a step
                  of the output's type.
"""
import sys

import numpy as np
import pytest

from oracle import logprob_oracle as O
from test_gpu_logprob import H24, NSUM, Bounds, DT, dev, host, same

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


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def inputs(rng, N, V, d, dtype, T):
    W = rng.standard_normal((V, d)) * (2.0 / np.sqrt(d))
    H = rng.standard_normal((N, d)) * 2
    ids = None
    if T:
        ids = rng.integers(-1, V + 1, (N, T)).astype(np.int32)
        if T > 2:
            ids[:, 2] = ids[:, 0]
        H += 2.0 * W[np.clip(ids[:, 0], 0, V - 1)]
    return dev(H, dtype), dev(W, dtype), ids


def check(ckl, N, V, d, dtype, T, mask=None, chunk=0, entropy=True, base=None):
    say(f"[case] head {dtype} N={N} V={V} d={d} T={T} mask={mask is not None} chunk={chunk} entropy={entropy} base={base}")
    rng = np.random.default_rng(N * 7 + V + d)
    tH, tW, ids = inputs(rng, N, V, d, dtype, T)
    H, W = host(tH), host(tW)
    tid = torch.from_numpy(ids).to("cuda:0") if T else None
    if T == 1:
        tid = tid[:, 0].contiguous()
    m = torch.from_numpy(mask).to("cuda:0") if mask is not None else None
    on = np.ones(N, bool) if mask is None else mask != 0
    out = ckl.head_logprobs(tH, tW, tid, mask=m, chunk=chunk)
    z = H @ W.T
    tz = (d + 8) * H24 * (np.abs(H) @ np.abs(W).T)
    E = tz.max(1)
    b = Bounds(z)
    assert not host(out.entropy)[~on].any() and not host(out.stats)[:, ~on].any()
    th = b.th + E * (b.p * np.abs(b.logp + b.H[:, None])).sum(1)
    same(host(out.entropy)[on], b.H[on], th[on], "entropy")
    st = host(out.stats)
    same(st[0][on], b.M[on], E[on], "M")
    same(st.sum(0)[on], (b.M + b.L)[on], (b.tl + E)[on], "log-normaliser")
    if T:
        got = host(out.logp).reshape(N, T)
        want = O.given(b.logp, ids)
        same(got[on], want[on], (b.of_logp(O.given(b.d, ids), want) + O.given(tz, ids) + E[:, None])[on], "logp")
        assert not got[~on].any()
    w = rng.standard_normal((N, T)).astype(np.float32) if T else None
    u = rng.standard_normal(N).astype(np.float32) if entropy else None
    dl = torch.from_numpy(w).to("cuda:0") if T else None
    if T == 1:
        dl = dl[:, 0].contiguous()
    tu = torch.from_numpy(u).to("cuda:0") if entropy else None
    kw = {}
    if base is not None:
        before = torch.randn(V, d, device="cuda:0") if base == "add" else torch.full((V, d), float("nan"), device="cuda:0")
        kw = {"dW": before.clone(), "accumulate": base == "add"}
    dH, dW = ckl.head_logprobs_bwd(tH, tW, tid, out.logp, out.entropy, out.stats, dl, tu, mask=m, chunk=chunk, **kw)
    G = O.logits_grad(z, ids, w, u)
    G[~on] = 0
    wt, wabs = O.weights(ids, w, V, N), O.weights(ids, np.abs(w) if T else None, V, N)
    U = np.abs(u)[:, None] if entropy else np.zeros((N, 1))
    c = np.abs(wt.sum(1) + (u * b.H if entropy else 0))[:, None]
    l = np.abs(b.logp)
    e_l = b.tl[:, None] + (b.d + l + b.L[:, None]) * H24 + tz + E[:, None]
    eG = b.p * ((c + U * l) * (e_l + (2 * l + 6) * H24) + U * e_l + U * th[:, None]
                + (T + 4) * H24 * (wabs.sum(1)[:, None] + U * (l + b.H[:, None]))) + T * H24 * wabs
    eG += 2.0 ** -126 * (1 + c + U * l)
    e = torch.finfo(DT[dtype]).eps / 2
    eG += e * (np.abs(G) + eG)
    eG[~on] = 0
    aG = np.abs(G) + eG
    want = G @ W
    bound = eG @ np.abs(W) + (V + 16) * H24 * (aG @ np.abs(W))
    same(host(dH), want, bound + e * (np.abs(want) + bound), "dH")
    assert not host(dH)[~on].any()
    want = G.T @ H
    bound = eG.T @ np.abs(H) + (N + 16) * H24 * (aG.T @ np.abs(H))
    if base == "add":
        want = want + host(before)
        bound = bound + 2 * H24 * np.abs(want)
    ew = torch.finfo(dW.dtype).eps / 2
    assert dW.dtype == (torch.float32 if base is not None else DT[dtype])
    same(host(dW), want, bound + ew * (np.abs(want) + bound), "dW")
    return out, dH, dW


SIZES = [(1, 1, 8), (1, 300, 64), (5, 127, 8), (3, 129, 24), (64, 1000, 72), (257, 513, 136), (300, 2000, 256),
         (2, 5003, 40), (40, 640, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d", SIZES)
def test_sizes(ckl, dtype, N, V, d):
    for T in (1, 0, 3):
        check(ckl, N, V, d, dtype, T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("base", [None, "own", "add"])
def test_chunks_and_masks(ckl, dtype, base):
    rng = np.random.default_rng(8)
    mask = (rng.random(600) < 0.7).astype(np.uint8)
    mask[256:512] = 0  # a chunk without a row
    for m in (None, mask):
        check(ckl, 600, 700, 72, dtype, 2, mask=m, chunk=256, base=base)
        check(ckl, 600, 700, 72, dtype, 1, mask=m, base=base, entropy=False)
    check(ckl, 70, 300, 64, dtype, 1, mask=np.zeros(70, np.uint8), base=base)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(ckl, dtype):
    # two and more chunks of thousands of rows, the last one short; many rows under few columns
    check(ckl, 8200, 200, 16, dtype, 1, chunk=4096)
    check(ckl, 9000, 130, 24, dtype, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d", [(500, 8000, 72), (600, 40000, 64), (40, 40000, 1032), (5000, 200, 2056), (2500, 700, 1032)])
def test_tiles(ckl, dtype, N, V, d):
    # products of 64, 128 and 256 wide tiles: the logits', dH's and dW's
    check(ckl, N, V, d, dtype, 1)


@pytest.mark.parametrize("T", [0, 1, 2])
def test_a_last_turn_of_smaller_tiles(ckl, T):
    # 256 tiles of 256 x 256 and 300 ids more, which go in tiles of 64 by a launch of their own
    mask = np.ones(256, np.uint8)
    mask[100:140] = 0
    check(ckl, 256, 65836, 520, "bf16", T, mask=mask if T == 2 else None)


def test_few_rows_past_a_tile(ckl):
    # dH in tiles of 128 and many splits; dW rounded by all three tiles' epilogues, added over chunks
    check(ckl, 300, 20000, 520, "bf16", 1)
    check(ckl, 300, 700, 136, "bf16", 1, chunk=256)
    check(ckl, 600, 9000, 2056, "bf16", 1, chunk=256)


@pytest.mark.parametrize("T", [64, 2048])
def test_given_tokens(ckl, T):
    check(ckl, 5, 300, 64, "bf16", T)
    check(ckl, 5, 300, 64, "f32", T)


def test_agrees_with_the_logits_form(ckl):
    rng = np.random.default_rng(6)
    tH, tW, ids = inputs(rng, 50, 3000, 128, "f32", 2)
    tid = torch.from_numpy(ids).to("cuda:0")
    a = ckl.head_logprobs(tH, tW, tid)
    z = (tH.double() @ tW.double().t())
    b = ckl.logprobs(z.float(), tid)
    # z rounded to fp32 on one side, an fp32 sum of 128 products of magnitude below 40 on the other
    assert bool((a.logp - b.logp).abs().max() <= 2e-3) and bool((a.entropy - b.entropy).abs().max() <= 2e-3)


def test_chunking_changes_no_statistics(ckl):
    rng = np.random.default_rng(7)
    tH, tW, ids = inputs(rng, 700, 900, 64, "bf16", 1)
    tid = torch.from_numpy(ids[:, 0].copy()).to("cuda:0")
    a, b = ckl.head_logprobs(tH, tW, tid), ckl.head_logprobs(tH, tW, tid, chunk=256)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    w = torch.randn(700, device="cuda:0")
    g = [ckl.head_logprobs_bwd(tH, tW, tid, *a, w, w) for _ in range(2)]
    assert torch.equal(g[0][0], g[1][0]) and torch.equal(g[0][1], g[1][1])


def test_nan_stays_in_its_row(ckl):
    tH, tW = torch.randn(9, 64, device="cuda:0"), torch.randn(500, 64, device="cuda:0")
    ids = torch.arange(9, device="cuda:0", dtype=torch.int32)
    clean = ckl.head_logprobs(tH, tW, ids)
    tH[4, 3] = float("nan")
    out = ckl.head_logprobs(tH, tW, ids)
    keep = [i for i in range(9) if i != 4]
    assert bool(out.logp[4].isnan()) and bool(out.entropy[4].isnan())
    assert torch.equal(out.logp[keep], clean.logp[keep]) and torch.equal(out.entropy[keep], clean.entropy[keep])
    one = torch.ones(9, device="cuda:0")
    dH, dW = ckl.head_logprobs_bwd(tH, tW, ids, *out, one, one)
    assert bool(dH[4].isnan().all()) and bool(dH[keep].isfinite().all()) and bool(dW.isnan().any())
    mask = torch.ones(9, dtype=torch.bool, device="cuda:0")
    mask[4] = False
    out = ckl.head_logprobs(tH, tW, ids, mask=mask)
    dH, dW = ckl.head_logprobs_bwd(tH, tW, ids, *out, one, one, mask=mask)
    assert all(bool(t.isfinite().all()) for t in (*out, dH, dW)) and not dH[4].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 600])
def test_weights_of_minus_infinity(ckl, dtype, N):
    """Ids whose logits are all -inf, whole slices of them, weigh nothing, as if they were not there."""
    V, cut, d = 9000, 300, 64
    rng = np.random.default_rng(N)
    H, W = rng.standard_normal((N, d)), rng.standard_normal((V, d))
    H[:, 0] = 1.0
    W[:cut, 0] = -np.inf
    tH, tW = dev(H, dtype), dev(W, dtype)
    ids = rng.integers(0, V, (N, 2)).astype(np.int32)
    ids[:, 1] = rng.integers(0, cut, N)
    out = ckl.head_logprobs(tH, tW, torch.from_numpy(ids).to("cuda:0"))
    H, W = host(tH), host(tW)[cut:]
    z = H @ W.T
    tz = (d + 8) * H24 * (np.abs(H) @ np.abs(W).T)
    E = tz.max(1)
    b = Bounds(z)
    same(host(out.entropy), b.H, b.th + E * (b.p * np.abs(b.logp + b.H[:, None])).sum(1), "entropy")
    same(host(out.stats)[0], b.M, E, "M")
    rest = np.where(ids >= cut, ids - cut, -1)
    want = O.given(b.logp, rest)
    bound = b.of_logp(O.given(b.d, rest), want) + O.given(tz, rest) + E[:, None]
    same(host(out.logp), np.where(ids >= cut, want, -np.inf), bound, "logp")
    one = torch.ones(N, device="cuda:0")
    _, dW = ckl.head_logprobs_bwd(tH, tW, None, None, out.entropy, out.stats, None, one)
    assert not dW[:cut].any() and bool(dW.isfinite().all()) and bool(dW[cut:].any())
    # no token at all
    W = tW[:cut].clone()
    for T in (1, 2):
        tid = torch.zeros((N, T), dtype=torch.int32, device="cuda:0")
        tid[:, -1] = -1
        out = ckl.head_logprobs(tH, W, tid)
        want = torch.full((N, T), -float("inf"), device="cuda:0")
        want[:, -1] = 0
        assert torch.equal(out.logp, want) and not out.entropy.any()
        assert bool((out.stats[0] == -float("inf")).all()) and not out.stats[1].any()
        tid.zero_()
        out = ckl.head_logprobs(tH, W, tid)
        _, dW = ckl.head_logprobs_bwd(tH, W, tid, *out, torch.ones(N, T, device="cuda:0"), one)
        assert not dW.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_certain_token_is_not_above_one(ckl, dtype):
    rng = np.random.default_rng(3)
    W = rng.standard_normal((700, 520))
    ids = rng.integers(0, 700, 300).astype(np.int32)
    tW = dev(W, dtype)
    out = ckl.head_logprobs(dev(W[ids], dtype), tW, torch.from_numpy(ids).to("cuda:0"))
    # its logit, sum W^2, is some 400 above any other, so logp is 0 but for its two sums' errors
    least = -2 * (520 + 8) * H24 * (host(tW) ** 2).sum(1).max()
    assert bool((out.logp <= 0).all()) and bool((out.logp >= least).all()) and bool((out.entropy >= 0).all())


def test_no_rows(ckl):
    W = torch.randn(50, 64, device="cuda:0").to(torch.bfloat16)
    H = torch.empty(0, 64, device="cuda:0", dtype=torch.bfloat16)
    ids = torch.empty(0, dtype=torch.int32, device="cuda:0")
    out = ckl.head_logprobs(H, W, ids)
    assert out.logp.shape == (0,) and out.stats.shape == (2, 0)
    dH, dW = ckl.head_logprobs_bwd(H, W, ids, *out, torch.empty(0, device="cuda:0"))
    assert dH.shape == (0, 64) and dW.dtype == torch.bfloat16 and not dW.any()
    before = torch.ones(50, 64, device="cuda:0")
    ckl.head_logprobs_bwd(H, W, ids, *out, torch.empty(0, device="cuda:0"), dW=before, accumulate=True)
    assert bool((before == 1).all())


def test_autograd(ckl):
    rng = np.random.default_rng(11)
    tH, tW, ids = inputs(rng, 60, 400, 72, "bf16", 1)
    tid = torch.from_numpy(ids[:, 0].copy()).to("cuda:0")
    H, W = tH.clone().requires_grad_(), tW.t().contiguous().t().requires_grad_()
    w, u = torch.randn(60, device="cuda:0"), torch.randn(60, device="cuda:0")
    out = ckl.head_logprobs(tH, tW, tid)
    for use in ("both", "logp", "entropy"):
        H.grad = W.grad = None
        logp, ent = ckl.head_token_logprobs(H, W, tid)
        loss = {"both": lambda: (logp * w + ent * u).sum(), "logp": lambda: (logp * w).sum(),
                "entropy": lambda: (ent * u).sum()}[use]()
        loss.backward()
        given = use != "entropy"
        want = ckl.head_logprobs_bwd(tH, tW, tid if given else None, out.logp if given else None, out.entropy, out.stats,
                                     w if given else None, u if use != "logp" else None)
        assert torch.equal(H.grad, want[0]) and torch.equal(W.grad, want[1])


def test_captured_and_two_streams(ckl):
    rng = np.random.default_rng(12)
    tH, tW, ids = inputs(rng, 300, 800, 64, "bf16", 1)
    tid = torch.from_numpy(ids[:, 0].copy()).to("cuda:0")
    mask = torch.rand(300, device="cuda:0") < 0.8
    m8 = mask.to(torch.uint8)
    w, u = torch.randn(300, device="cuda:0"), torch.randn(300, device="cuda:0")

    def step():
        out = ckl.head_logprobs(tH, tW, tid, mask=m8)
        return *out, *ckl.head_logprobs_bwd(tH, tW, tid, *out, w, u, mask=m8)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
    for i in range(4):
        tH.normal_()
        m8.copy_((torch.rand(300, device="cuda:0") < 0.5).to(torch.uint8))
        for g, _ in graphs:
            g.replay()
        want = step()
        torch.cuda.synchronize()
        for _, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want)), i
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(step())
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_a_training_step_with_the_loss(ckl):
    """The end of a block with dropout, the distillation loss and a policy's term at the same head, tied gradients."""
    rng = np.random.default_rng(13)
    N, V, d, K = 200, 1000, 64, 20
    t = {k: dev(rng.standard_normal(s), "f32") for k, s in
         {"y": (N, d), "r": (N, d), "w_pre": (d,), "w_post": (d,), "gate": (d,), "W": (V, d)}.items()}
    ids = np.stack([rng.permutation(V)[:K] for _ in range(N)]).astype(np.int32)
    tl = rng.standard_normal((N, K)).astype(np.float32)
    tids, ttl = torch.from_numpy(ids).to("cuda:0"), torch.from_numpy(tl).to("cuda:0")
    tok = tids[:, 0].contiguous()
    adv, u = torch.randn(N, device="cuda:0") / N, torch.full((N,), 0.01 / N, device="cuda:0")
    how = {"gate": t["gate"], "scale": 0.5, "p": 0.1, "seed": 21, "offset": 2}
    ro, x, stats = ckl.add_norm(t["y"], t["r"], t["w_pre"], t["w_post"], stats=True, **how)
    loss, dx, dW = ckl.fwd_bwd(x, t["W"], tids, ttl)
    out = ckl.head_logprobs(x, t["W"], tok)
    dx2, same_dW = ckl.head_logprobs_bwd(x, t["W"], tok, *out, adv, u, dW=dW, accumulate=True)
    assert same_dW is dW
    dy, dr, dw_post, dw_pre, dgate = ckl.add_norm_bwd(t["y"], t["r"], t["w_pre"], t["w_post"], stats, dx + dx2, None, **how)
    # the same step by torch's autograd in float64, with the dropout's own factors
    from oracle import residual_oracle as R

    f = torch.from_numpy(0.5 * R.factors(N * d, 0.1, 21, 2).reshape(N, d)).to("cuda:0")
    v = {k: a.double().requires_grad_() for k, a in t.items()}
    unit = lambda a: a / (a.pow(2).mean(1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    xx = unit(v["r"] + f * v["gate"] * v["w_post"] * unit(v["y"])) * v["w_pre"]
    logp = torch.log_softmax(xx @ v["W"].t(), 1)
    pt = torch.softmax(ttl.double(), 1)
    kl = (pt * (pt.log() - logp.gather(1, tids.long()))).sum(1).mean()
    total = kl + (adv.double() * logp.gather(1, tok.long()[:, None])[:, 0]).sum() - (u.double() * (logp.exp() * logp).sum(1)).sum()
    total.backward()
    # fp32 throughout: logits within (64 + 8) 2^-24 of a sum of magnitudes below 200, so l within 1.7e-3 and p within
    # that relative; sums of such errors over V and N stay within that share of the gradient's norm
    for got, name in ((dy, "y"), (dr, "r"), (dw_post, "w_post"), (dw_pre, "w_pre"), (dgate, "gate"), (dW, "W")):
        want = v[name].grad
        assert float((got.double() - want).norm() / want.norm()) <= 2e-3, name
    assert abs(loss.item() - kl.item()) <= 2e-3 * abs(kl.item())


def test_refusals(ckl):
    H, W = torch.randn(4, 64, device="cuda:0"), torch.randn(30, 64, device="cuda:0")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    for bad in ({"H": H.cpu()}, {"H": H.half()}, {"H": H[:, :32]}, {"W": W.bfloat16()}, {"W": W[:, :32]}, {"W": W.cpu()},
                {"H": H.t().contiguous().t()}, {"ids": ids.long()}, {"ids": ids[:2]}, {"mask": ids[:1]}, {"H": H[0]}):
        with pytest.raises(ValueError):
            ckl.head_logprobs(**{"H": H, "W": W, "ids": ids, **bad})
    with pytest.raises(ckl.CklError):
        ckl.head_logprobs(H[:, :60].contiguous(), W[:, :60].contiguous(), ids)
    with pytest.raises(ckl.CklError):
        ckl.head_logprobs(H, W, ids, chunk=-1)
    out = ckl.head_logprobs(H, W, ids)
    w = torch.ones(4, device="cuda:0")
    ok = {"H": H, "W": W, "ids": ids, "logp": out.logp, "entropy": out.entropy, "stats": out.stats, "dlogp": w}
    b16 = {"H": H.bfloat16(), "W": W.bfloat16()}
    for bad in ({"dlogp": None}, {"logp": None}, {"stats": None}, {"entropy": None, "dentropy": w}, {"dentropy": w[:2]},
                {"accumulate": True}, {"dW": W[:5]}, {"dW": W.bfloat16()}, {"logp": out.logp[:2]}, {"ids": None},
                {**b16, "dW": W.bfloat16(), "accumulate": True}):
        with pytest.raises(ValueError):
            ckl.head_logprobs_bwd(**{**ok, **bad})
    leaf = H.clone().requires_grad_()
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(g):
            ckl.head_token_logprobs(leaf, W, ids)
