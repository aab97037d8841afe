"""Log-probabilities of given tokens, entropy and alternatives from logits on the GPU, and their gradient, against the
float64 oracle.

Tolerances, with h = 2^-24 (half a step of fp32), d = M - z, L the log of the sum, to first order:
  a logit's share e = exp(z - m) about a reference m at most 8 below M: (2 (d + 8) + 4) h relative.  Sums: a thread adds
  at most V / 64 terms for V <= 1,024, V / 256 up to 8,192, V / 1,024 or V / (256 slices) beyond, so under 300 here, then
  under 30 across threads, and 3 a move of the reference (at most one a vector of 8; under 40 matter, since each lets
  what was before weigh exp(-8)): n = 400 in all.  With t1 = sum p d, t2 = sum p d^2:
    L         (n + 2 (t1 + 8) + 4 + 2 L) h
    logp      L's, and (d + |logp| + L) h
    entropy   L's, and (2 t2 + 40 (t1 + 8) + (2 n + 8) (t1 + 8) + 2 L) h
  gradient    half a step of the output, and, with dl = L's + (d + |l| + L) h the error of l = log p and c = sum w + u H:
              p [(|c| + |u l|) (dl + (2 |l| + 6) h) + |u| dl + |u| entropy's + (T + 4) h (sum |w| + |u| (|l| + H))] + T h |w|,
              and what a p below 2^-126, which is taken as 0, is multiplied with: 2^-126 (1 + |c| + |u l|)
  alternatives' ids are exact.
"""
import sys

import numpy as np
import pytest

from oracle import logprob_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
H24 = 2.0 ** -24
NSUM = 400


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


def host(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


class Bounds:
    def __init__(self, z):
        self.M, self.L, self.H, self.p, self.logp = O.row_stats(z)
        with np.errstate(invalid="ignore"):
            d = np.where(self.p > 0, np.where(np.isfinite(self.M), self.M, 0)[:, None] - z, 0.0)
        self.d = d
        t1, t2 = (self.p * d).sum(1) + 8, (self.p * d * d).sum(1)
        self.tl = (NSUM + 2 * t1 + 4 + 2 * self.L) * H24
        self.th = self.tl + (2 * t2 + 40 * t1 + (2 * NSUM + 8) * t1 + 2 * self.L) * H24

    def of_logp(self, d, logp):
        with np.errstate(invalid="ignore"):
            r = self.tl[:, None] + (d + np.abs(logp) + self.L[:, None]) * H24
        return np.where(np.isfinite(logp), r, 0.0)


def same(got, want, bound, what):
    fin = np.isfinite(want)
    np.testing.assert_array_equal(got[~fin], want[~fin], err_msg=what)
    err = np.abs(got[fin] - want[fin])
    b = np.broadcast_to(bound, want.shape)[fin]
    assert np.all(err <= b), (what, float(np.max(err - b)), float(np.max(err)))


def make(rng, N, V, kind):
    z = 2 * rng.standard_normal((N, V))
    if kind == "peaked":
        z[np.arange(N), rng.integers(0, V, N)] += 12
    elif kind == "banned":
        z[:, rng.random(V) < 0.3] = -np.inf
        z[:, 0] = 1.0
    elif kind == "constant":
        z[:] = -1.5
    elif kind == "few values":
        z = np.round(z / 2)
    elif kind == "lowest":  # masked with the type's lowest value, some rows wholly
        z[:, rng.random(V) < 0.5] = -3.3895313892515355e38
        z[::3] = -3.3895313892515355e38
    elif kind == "rising":
        z = np.sort(z, 1) * 20
    elif kind == "zeros":
        z = np.where(rng.random((N, V)) < 0.5, 0.0, -0.0)
    return z


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to("cuda:0").to(DT[dtype])


def check(ckl, z, dtype, T, top, rng, pad=0, mask=None, grad=True):
    N, V = z.shape
    say(f"[case] logprobs {dtype} N={N} V={V} T={T} top={top} pad={pad} mask={mask is not None}")
    x = dev(np.concatenate([z, np.full((N, pad), 99.0)], 1) if pad else z, dtype)[:, :V]
    z = host(x)
    ids = None
    if T:
        ids = rng.integers(-1, V + 1, (N, T)).astype(np.int32)
        if T > 2:
            ids[:, 2] = ids[:, 0]
        ids[0, 0] = np.iinfo(np.int32).min if N > 1 else ids[0, 0]
    tid = torch.from_numpy(ids).to("cuda:0") if T else None
    if T == 1:
        tid = tid[:, 0].contiguous()
    m = torch.from_numpy(mask).to("cuda:0") if mask is not None else None
    out = ckl.logprobs(x, tid, top=top, mask=m)
    on = np.ones(N, bool) if mask is None else mask != 0
    b = Bounds(z)
    assert not host(out.entropy)[~on].any() and not host(out.stats)[:, ~on].any()
    same(host(out.entropy)[on], b.H[on], b.th[on], "entropy")
    np.testing.assert_array_equal(host(out.stats)[0][on], b.M[on])
    same(host(out.stats)[1][on], b.L[on], b.tl[on], "L")
    if T:
        got = host(out.logp).reshape(N, T)
        want = O.given(b.logp, ids)
        same(got[on], want[on], b.of_logp(np.abs(np.where(np.isfinite(O.given(b.d, ids)), O.given(b.d, ids), 0)), want)[on],
             "logp")
        assert not got[~on].any()
    else:
        assert out.logp is None
    if top:
        wid, wlp = O.top(z, b.logp, top)
        wid[~on], wlp[~on] = -1, 0.0
        np.testing.assert_array_equal(host(out.top_ids), wid)
        same(host(out.top_logp)[on], wlp[on], b.of_logp(np.abs(np.where(np.isfinite(wlp), wlp, 0)) + b.L[:, None], wlp)[on],
             "top")
        assert not host(out.top_logp)[~on].any()
    if not grad:
        return out
    w = rng.standard_normal((N, T)).astype(np.float32) if T else None
    u = rng.standard_normal(N).astype(np.float32)
    dl = torch.from_numpy(w).to("cuda:0") if T else None
    if T == 1:
        dl = dl[:, 0].contiguous()
    g = ckl.logprobs_bwd(x, tid, out.entropy, out.stats, dl, torch.from_numpy(u).to("cuda:0"), mask=m)
    want = O.logits_grad(z, ids, w, u.astype(np.float64))
    want[~on] = 0
    wt, wabs = O.weights(ids, w, V, N), O.weights(ids, np.abs(w) if T else None, V, N)
    l = np.where(b.p > 0, b.logp, 0.0)
    e_l = b.tl[:, None] + (b.d + np.abs(l) + b.L[:, None]) * H24
    c = np.abs(wt.sum(1) + u * b.H)[:, None]
    U, A = np.abs(u)[:, None], wabs.sum(1)[:, None]
    bound = b.p * ((c + U * np.abs(l)) * (e_l + (2 * np.abs(l) + 6) * H24) + U * e_l + U * b.th[:, None]
                   + (T + 4) * H24 * (A + U * (np.abs(l) + b.H[:, None]))) + T * H24 * wabs
    bound += 2.0 ** -126 * (1 + c + U * np.abs(l))  # a p below the smallest normal number is 0
    rounded = lambda want: bound + torch.finfo(DT[dtype]).eps / 2 * (np.abs(want) + bound)  # noqa: E731
    same(host(g), want, rounded(want), "gradient")
    if pad == 0:  # in place
        y = x.clone()
        assert ckl.logprobs_bwd(y, tid, out.entropy, out.stats, dl, torch.from_numpy(u).to("cuda:0"), mask=m, out=y) is y
        assert torch.equal(y, g)
    if T:  # without the entropy's gradient
        g = ckl.logprobs_bwd(x, tid, None, out.stats, dl, None, mask=m)
        want = O.logits_grad(z, ids, w, None)
        want[~on] = 0
        same(host(g), want, rounded(want), "gradient of logp")  # the output's half step goes by its own value
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V", [(1, 1), (2, 7), (3, 8), (5, 9), (300, 65), (4, 1000), (3, 1024), (3, 1025), (2, 8192),
                                 (300, 8193), (3, 8193), (1, 40001), (70, 16400), (260, 10000)])
def test_sizes(ckl, dtype, N, V):
    rng = np.random.default_rng(N + V)
    for T, top in ((1, min(5, V)), (0, 0), (3, min(20, V))):
        check(ckl, make(rng, N, V, "peaked"), dtype, T, top, rng)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["bulk", "banned", "constant", "few values", "lowest", "rising", "zeros"])
@pytest.mark.parametrize("N,V", [(6, 500), (6, 4099), (3, 20011), (256, 9000)])
def test_kinds(ckl, dtype, kind, N, V):
    rng = np.random.default_rng(V)
    check(ckl, make(rng, N, V, kind), dtype, 2, 20, rng)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [1, 47, 48, 49, 128, 129, 500, 512])
@pytest.mark.parametrize("kind", ["bulk", "few values"])
def test_alternatives(ckl, dtype, top, kind):
    rng = np.random.default_rng(top)
    for N, V in ((3, 600), (2, 6000), (256, 8500), (2, 30000), (1, 100003)):
        check(ckl, make(rng, N, V, kind), dtype, 0, top, rng, grad=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 64, 257, 2048])
def test_given_tokens(ckl, dtype, T):
    rng = np.random.default_rng(T)
    check(ckl, make(rng, 3, 9001, "peaked"), dtype, T, 0, rng)
    check(ckl, make(rng, 2, 3, "bulk"), dtype, T, 3, rng)  # every token many times


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_masks(ckl, dtype):
    rng = np.random.default_rng(9)
    for N, V, pad in ((4, 1001, 3), (5, 20000, 1), (300, 333, 7)):
        mask = (rng.random(N) < 0.6).astype(np.uint8)
        check(ckl, make(rng, N, V, "bulk"), dtype, 2, 6, rng, pad=pad, mask=mask)
    check(ckl, make(rng, 4, 300, "bulk"), dtype, 1, 2, rng, mask=np.zeros(4, np.uint8))


def test_masked_rows_are_not_read_into_anything(ckl):
    x = torch.randn(6, 12000, device="cuda:0")
    x[1], x[4] = float("nan"), float("inf")
    keep = torch.tensor([1, 0, 1, 1, 0, 1], device="cuda:0", dtype=torch.bool)
    ids = torch.zeros(6, dtype=torch.int32, device="cuda:0")
    out = ckl.logprobs(x, ids, top=3, mask=keep)
    assert all(bool(t.isfinite().all()) for t in (out.logp, out.entropy, out.stats, out.top_logp))
    g = ckl.logprobs_bwd(x, ids, out.entropy, out.stats, torch.ones(6, device="cuda:0"), torch.ones(6, device="cuda:0"),
                         mask=keep)
    assert bool(g.isfinite().all()) and not g[[1, 4]].any()


@pytest.mark.parametrize("V", [300, 5000, 30000])
def test_nan_inf_and_empty_rows(ckl, V):
    x = torch.randn(5, V, device="cuda:0")
    x[0, V // 2] = float("nan")
    x[1, V - 1] = float("inf")
    x[2] = -float("inf")
    x[3, 1:] = -float("inf")
    ids = torch.tensor([3, V - 1, 0, 0, 1], dtype=torch.int32, device="cuda:0")
    out = ckl.logprobs(x, ids, top=4)
    nan = [bool(v) for v in out.logp.isnan()]
    assert nan == [True, True, False, False, False]
    assert [bool(v) for v in out.entropy.isnan()] == nan
    assert out.logp[2].item() == -float("inf") and out.entropy[2].item() == 0.0
    assert out.logp[3].item() == 0.0 and out.entropy[3].item() == 0.0
    assert out.top_ids[1, 0].item() == V - 1 and V // 2 not in out.top_ids[0].tolist()
    assert out.top_ids[2].tolist() == [-1] * 4 and bool((out.top_logp[2] == -float("inf")).all())
    assert out.top_ids[3].tolist() == [0, -1, -1, -1] and out.top_logp[3, 0].item() == 0.0
    one = torch.ones(5, device="cuda:0")
    g = ckl.logprobs_bwd(x, ids, out.entropy, out.stats, one, one)
    assert bool(g[0].isnan().any()) and not g[2].any() and bool(g[3:].isfinite().all()) and g[3, 0].item() == 0.0


def test_far_offsets(ckl):
    """Rows that start past 2^32 bytes of the logits."""
    V, N = 201088, 12000
    x = torch.zeros(N, V, device="cuda:0", dtype=torch.bfloat16)
    x[N - 1, 123456] = 5.0
    out = ckl.logprobs(x, torch.full((N,), 123456, dtype=torch.int32, device="cuda:0"), top=2)
    want = 5.0 - np.log(V - 1 + np.exp(5.0))
    assert abs(out.logp[N - 1].item() - want) <= 1e-5 * abs(want)  # 400 roundings of 2^-24
    assert out.top_ids[N - 1].tolist() == [123456, 0] and out.top_ids[0].tolist() == [0, 1]
    g = ckl.logprobs_bwd(x, None, out.entropy, out.stats, None, None, out=x)
    assert not g.any()


def test_no_rows(ckl):
    x = torch.empty(0, 50, device="cuda:0")
    out = ckl.logprobs(x, torch.empty(0, 3, dtype=torch.int32, device="cuda:0"), top=2)
    assert out.logp.shape == (0, 3) and out.top_ids.shape == (0, 2) and out.stats.shape == (2, 0)
    assert ckl.logprobs_bwd(x, None, out.entropy, out.stats).shape == (0, 50)


def test_sampled_tokens_log_probability(ckl):
    """A decode step: the drawn token's report agrees with the sampler's."""
    g = torch.Generator(device="cuda:0")
    g.manual_seed(4)
    x = (3 * torch.randn(33, 32000, device="cuda:0", generator=g)).to(torch.bfloat16)
    ids, logp = ckl.sample(x, torch.rand(33, device="cuda:0", generator=g))
    out = ckl.logprobs(x, ids, top=1)
    assert bool((out.logp - logp).abs().max() <= 1e-4)  # (400 + 2 x 30) 2^-24 x 2, and the sampler's own
    assert torch.equal(out.top_ids[:, 0], x.float().argmax(1).to(torch.int32))
    greedy, _ = ckl.sample(x, torch.rand(33, device="cuda:0"), temperature=0)
    assert torch.equal(out.top_ids[:, 0], greedy)


def test_same_bits_and_two_streams(ckl):
    x = torch.randn(40, 50000, device="cuda:0").to(torch.bfloat16)
    ids = torch.randint(0, 50000, (40, 3), device="cuda:0").to(torch.int32)
    first = ckl.logprobs(x, ids, top=30)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(ckl.logprobs(x, ids, top=30))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, first))


def test_captured(ckl):
    x = torch.randn(7, 30000, device="cuda:0")
    ids = torch.randint(0, 30000, (7, 2), device="cuda:0").to(torch.int32)
    w, u = torch.randn(7, 2, device="cuda:0"), torch.randn(7, device="cuda:0")

    def step():
        out = ckl.logprobs(x, ids, top=9)
        return *out, ckl.logprobs_bwd(x, ids, out.entropy, out.stats, w, u)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):  # two graphs hold a workspace each
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
    for i in range(4):
        x.normal_()
        for g, got in graphs:
            g.replay()
        want = step()
        torch.cuda.synchronize()
        for _, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_autograd(ckl):
    rng = np.random.default_rng(2)
    z = make(rng, 9, 700, "peaked")
    x = dev(z, "f32").requires_grad_()
    ids = torch.from_numpy(rng.integers(-1, 700, (9, 2)).astype(np.int32)).to("cuda:0")
    w, u = torch.randn(9, 2, device="cuda:0"), torch.randn(9, device="cuda:0")
    for use_w, use_u in ((True, True), (True, False), (False, True)):
        x.grad = None
        logp, ent = ckl.token_logprobs(x, ids)
        ((logp * w).sum() * use_w + (ent * u).sum() * use_u if use_w and use_u else (logp * w).sum() if use_w
         else (ent * u).sum()).backward()
        out = ckl.logprobs(x.detach(), ids)
        got = ckl.logprobs_bwd(x.detach(), ids if use_w else None, out.entropy, out.stats, w if use_w else None,
                               u if use_u else None)
        assert torch.equal(x.grad, got)
    t = x.detach().t().contiguous().t().requires_grad_()  # columns adjacent: copied
    ckl.token_logprobs(t, ids)[0].sum().backward()
    assert t.grad.shape == t.shape


def test_refusals(ckl):
    x = torch.randn(4, 60, device="cuda:0")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    for bad in ({"logits": x.cpu()}, {"logits": x.half()}, {"logits": x[0]}, {"logits": x.t()}, {"ids": ids.long()},
                {"ids": ids[:3]}, {"ids": ids.cpu()}, {"ids": ids.view(4, 1, 1)}, {"mask": ids[:2]}, {"mask": ids.cpu()},
                {"top": -1}, {"top": 61}):
        with pytest.raises(ValueError):
            ckl.logprobs(**{"logits": x, "ids": ids, **bad})
    big = torch.randn(2, 600, device="cuda:0")
    with pytest.raises(ckl.CklError):
        ckl.logprobs(big, top=513)
    with pytest.raises(ckl.CklError):
        ckl.logprobs(big, torch.zeros(2, 2049, dtype=torch.int32, device="cuda:0"))
    out = ckl.logprobs(x, ids)
    w = torch.ones(4, device="cuda:0")
    for bad in ({"dlogp": None}, {"ids": None}, {"dlogp": w.double()}, {"dentropy": w[:2]}, {"stats": None},
                {"entropy": None, "dentropy": w}, {"out": x[:2]}, {"stats": out.stats[0]}):
        with pytest.raises(ValueError):
            ckl.logprobs_bwd(**{"logits": x, "ids": ids, "entropy": out.entropy, "stats": out.stats, "dlogp": w, **bad})
    rows = torch.randn(60, device="cuda:0").expand(4, 60)  # one row for all: read, never written
    ckl.logprobs(rows, ids)
    with pytest.raises(ValueError):
        ckl.logprobs_bwd(rows, ids, out.entropy, out.stats, w, out=rows)
    leaf = x.clone().requires_grad_()
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(g):
            ckl.token_logprobs(leaf, ids)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rising", "falling", "one slice", "level", "few above -inf"])
@pytest.mark.parametrize("top", [20, 128, 400])
def test_alternatives_of_few_rows_in_few_slices(ckl, dtype, kind, top):
    """Rows split over workgroups whose alternatives lie side by side, are all equal, or are too few."""
    N, V = 3, 100003
    say(f"[case] few rows {dtype} {kind} top={top}")
    rng = np.random.default_rng(top)
    z = {"rising": lambda: np.tile(np.linspace(-3, 8, V), (N, 1)), "falling": lambda: np.tile(np.linspace(8, -3, V), (N, 1)),
         "one slice": lambda: rng.standard_normal((N, V)), "level": lambda: np.full((N, V), 1.5),
         "few above -inf": lambda: np.full((N, V), -np.inf)}[kind]()
    if kind == "one slice":
        z[:, 50000:50600] += 20
    if kind == "few above -inf":
        z[:, rng.permutation(V)[:top - 1]] = rng.standard_normal(top - 1)
    x = dev(z, dtype)
    out = ckl.logprobs(x, None, top=top)
    h = host(x)
    b = Bounds(h)
    for n in range(N):
        order = np.lexsort((np.arange(V), -h[n]))[:top]
        ids = np.where(np.isfinite(h[n][order]), order, -1)
        np.testing.assert_array_equal(host(out.top_ids)[n], ids)
        want = np.where(ids >= 0, b.logp[n][order], -np.inf)
        same(host(out.top_logp)[n], want, b.of_logp(b.d[n][order], want)[n], "top_logp")
