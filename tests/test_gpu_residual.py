"""The residual's norms and dropout on the GPU against the float64 oracle.

Tolerances, with h = 2^-24 (half a step of fp32) and e = half a step of the output's type, to first order:
  dropout   one fp32 product rounded once: compared bit for bit.
  r_out     e |r_out| + 64 h M, M = |r| + |branch|.  1 / rms: at most 24 sums in a lane, 6 across lanes, 16 across
            waves, the mean, eps, root and quotient halve the sums' share (23 h) and add 4; five more products and
            the sum with r: under 40.
  x         e |x| + 192 h (w / rms) M': its r_out's 64 h M, the same of 1 / rms(r_out) through the row's norm of M, 40
            of its own.  M' = M + |r_out| (norm of M / norm of r_out).
  gradients e |g| + 512 h M with the oracle's magnitudes: means of up to 46 sums over terms of under 100 h each,
            three of them in dy's, products beside them.
  sums over rows of n terms: (n + 100 + 512) h M: n - 1 sums at most in a workgroup, under 80 across them.
A magnitude's own error (second order) is far below what these counts leave."""
import sys

import numpy as np
import pytest

from oracle import residual_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
H = 2.0 ** -24


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


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to("cuda:0").to(DT[dtype])


def host(t):
    return None if t is None else t.double().cpu().numpy()


def near(got, want, mag, count, dtype, what):
    e = torch.finfo(DT[dtype]).eps / 2
    err, bound = np.abs(host(got) - want), e * np.abs(want) + count * H * mag
    assert np.all(err <= bound), (what, float(np.max(err / np.maximum(bound, 1e-300))))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2049, 8192, 65537])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.7, 1.0])
def test_drop_is_exact(ckl, dtype, n, p):
    say(f"[case] drop {dtype} n={n} p={p}")
    x = torch.randn(n + 3, device="cuda:0").to(DT[dtype])[3:]  # not aligned to 16 bytes
    if n > 100:
        x[5], x[6], x[7] = float("inf"), float("nan"), -float("inf")
    seed, offset = (1 << 63) + 12345, (1 << 40) + 7
    f = torch.from_numpy(O.factors(n, p, seed, offset)).to("cuda:0").float()
    want = torch.where(f != 0, x.float() * f, torch.zeros((), device="cuda:0")).to(DT[dtype])
    got = ckl.drop(x, p, seed, offset)
    same = (got == want) | (got.isnan() & want.isnan())
    assert bool(same.all())
    assert got.isnan().sum() == want.isnan().sum()
    at = torch.tensor([offset], device="cuda:0")
    assert torch.equal(ckl.drop(x, p, seed, at).nan_to_num(5.0), got.nan_to_num(5.0))
    y = x.clone()
    ckl.drop(y, p, seed, offset, out=y)
    assert torch.equal(y.nan_to_num(5.0), got.nan_to_num(5.0))


def test_drop_of_none(ckl):
    assert ckl.drop(torch.empty((0, 5), device="cuda:0"), 0.5, 1).shape == (0, 5)


def run(ckl, dtype, N, d, post, pre, gate, p, grads=("dx", "dr"), scale=0.7, eps=1e-6, seed=77, offset=5, lead=None):
    rng = np.random.default_rng(N * 31 + d)
    t = {"y": dev(rng.standard_normal((N, d)) * 2, dtype), "r": dev(rng.standard_normal((N, d)) * 3, dtype),
         "w_pre": dev(1 + 0.3 * rng.standard_normal(d), dtype) if pre else None,
         "w_post": dev(1 + 0.3 * rng.standard_normal(d), dtype) if post else None,
         "gate": {"none": None, "vector": dev(rng.standard_normal(d), dtype),
                  "full": dev(rng.standard_normal((N, d)), dtype)}[gate],
         "dx": dev(rng.standard_normal((N, d)), dtype) if pre and "dx" in grads else None,
         "dr": dev(rng.standard_normal((N, d)), dtype) if "dr" in grads else None}
    shaped = lambda v: v if v is None or lead is None or v.dim() == 1 else v.view(*lead, d)  # noqa: E731
    how = {"gate": shaped(t["gate"]), "scale": scale, "p": p, "seed": seed, "offset": offset, "eps": eps}
    ro, x, stats = ckl.add_norm(shaped(t["y"]), shaped(t["r"]), t["w_pre"], t["w_post"], stats=True, **how)
    g = ckl.add_norm_bwd(shaped(t["y"]), shaped(t["r"]), t["w_pre"], t["w_post"], stats, shaped(t["dx"]),
                         shaped(t["dr"]), **how) if grads else None
    return t, ro, x, stats, g


def check(ckl, dtype, N, d, post, pre, gate, p, **kw):
    say(f"[case] add_norm {dtype} N={N} d={d} post={post} pre={pre} gate={gate} p={p} {kw}")
    eps = kw.get("eps", 1e-6)
    t, ro, x, stats, g = run(ckl, dtype, N, d, post, pre, gate, p, **kw)
    v = {k: host(a) for k, a in t.items()}
    f = float(np.float32(kw.get("scale", 0.7))) * (O.factors(N * d, p, 77, 5).reshape(N, d) if p else np.ones((N, d)))
    wro, wx, mag, inv1, inv2 = O.add_norm(v["y"], v["r"], v["w_pre"], v["w_post"], v["gate"], f, float(np.float32(eps)))
    near(ro.view(N, d), wro, mag, 64, dtype, "r_out")
    if pre:
        norm = lambda a: np.sqrt((a * a).sum(1, keepdims=True))  # noqa: E731
        m = mag + np.abs(wro) * (norm(mag) / np.maximum(norm(wro), 1e-30))
        near(x.view(N, d), wx, np.abs(v["w_pre"]) * inv2 * m, 192, dtype, "x")
    else:
        assert x is None
    if g is None:
        return
    want = O.add_norm_grad(v["y"], v["r"], v["w_pre"], v["w_post"], v["gate"], f, float(np.float32(eps)), v["dx"], v["dr"])
    dy, dr, dw_post, dw_pre, dgate = g
    near(dr.view(N, d), *want["dr"], 512, dtype, "dr")
    near(dy.view(N, d), *want["dy"], 512, dtype, "dy")
    for name, got, there in (("dw_post", dw_post, post), ("dw_pre", dw_pre, pre), ("dgate", dgate, gate == "vector")):
        if there:
            assert got.dtype == torch.float32
            near(got, want[name][0].sum(0), want[name][1].sum(0), N + 612, "f32", name)
    if gate == "full":
        near(dgate.view(N, d), *want["dgate"], 512, dtype, "dgate")
    assert (dw_post is None) == (not post) and (dw_pre is None) == (not pre) and (dgate is None) == (gate == "none")


# rows of one lane up to the widest, both sides of every change of shape: rows side by side up to 512 elements, one or
# two vectors a lane from 1,024, workgroups of more than 512 threads from 4,096 or 8,192, two vectors of those from 8,192
SIZES = [(1, 8), (5, 16), (67, 24), (130, 64), (9, 512), (9, 520), (7, 1024), (7, 1032), (3, 1536), (3, 1544), (257, 2880),
         (3, 4096), (2, 4104), (3, 8192), (600, 8200), (2, 12288), (2, 12296), (3, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,d", SIZES)
def test_sizes(ckl, dtype, N, d):
    check(ckl, dtype, N, d, True, True, "vector", 0.2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gate", ["none", "vector", "full"])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_forms(ckl, dtype, post, pre, gate, p):
    check(ckl, dtype, 37, 200, post, pre, gate, p)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1032, 4104, 8200])
def test_wide_rows_with_their_own_gates(ckl, dtype, d):
    check(ckl, dtype, 5, d, True, True, "full", 0.2)
    check(ckl, dtype, 5, d, False, True, "none", 0.0)


@pytest.mark.parametrize("p", [1.0, 1 - 2.0 ** -18, 2.0 ** -18])
def test_everything_or_nothing_dropped(ckl, p):
    check(ckl, "f32", 21, 72, True, True, "vector", p)
    check(ckl, "bf16", 21, 72, True, True, "full", p)


@pytest.mark.parametrize("grads", [("dx",), ("dr",)])
def test_one_upstream_gradient(ckl, grads):
    check(ckl, "f32", 19, 72, True, True, "vector", 0.1, grads=grads)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(ckl, dtype):
    # more rows than workgroups in each shape of a row: several turns, the last one short
    check(ckl, dtype, 40001, 8, True, True, "vector", 0.0)
    check(ckl, dtype, 9001, 72, True, True, "vector", 0.0)


def test_numbers(ckl):
    check(ckl, "f32", 5, 64, True, True, "none", 0.0, scale=0.0)
    check(ckl, "f32", 5, 64, True, True, "none", 1.0)
    check(ckl, "f32", 5, 64, True, True, "none", 0.0, eps=0.5, scale=-2.0)
    check(ckl, "bf16", 12, 40, True, True, "full", 0.25, lead=(3, 4))


def test_rows_of_zeros(ckl):
    z = torch.zeros(3, 64, device="cuda:0")
    w = torch.ones(64, device="cuda:0")
    ro, x, stats = ckl.add_norm(z, z, w, w, stats=True)
    assert not ro.any() and not x.any()
    one = torch.ones_like(z)
    got = ckl.add_norm_bwd(z, z, w, w, stats, one, one)
    assert all(bool(g.isfinite().all()) for g in got[:4])
    # eps = 0: the formula's 0 / 0, in the row that has it and no other
    y = torch.randn(3, 64, device="cuda:0")
    y[1] = 0
    ro, x, _ = ckl.add_norm(y, z, w, None, eps=0.0)
    assert bool(x[1].isnan().all()) and bool(x[[0, 2]].isfinite().all())


def test_nan_stays_in_its_row(ckl):
    y, r, w = torch.randn(5, 48, device="cuda:0"), torch.randn(5, 48, device="cuda:0"), torch.ones(48, device="cuda:0")
    clean = ckl.add_norm(y, r, w, w)
    y[2, 3] = float("nan")
    ro, x, _ = ckl.add_norm(y, r, w, w)
    keep = [0, 1, 3, 4]
    assert bool(ro[2].isnan().all()) and torch.equal(ro[keep], clean[0][keep]) and torch.equal(x[keep], clean[1][keep])


def test_in_place_and_same_bits(ckl):
    t, ro, x, stats, g = run(ckl, "bf16", 300, 2880, True, True, "vector", 0.1)
    how = {"gate": t["gate"], "scale": 0.7, "p": 0.1, "seed": 77, "offset": 5}
    at = torch.tensor([5], device="cuda:0")
    for kw in ({}, {"offset": at}):
        again = ckl.add_norm(t["y"], t["r"], t["w_pre"], t["w_post"], stats=True, **{**how, **kw})
        assert all(torch.equal(a, b) for a, b in zip(again, (ro, x, stats)))
    gg = ckl.add_norm_bwd(t["y"], t["r"], t["w_pre"], t["w_post"], stats, t["dx"], t["dr"], **how)
    assert all(torch.equal(a, b) for a, b in zip(gg, g))
    r = t["r"].clone()
    got = ckl.add_norm(t["y"], r, t["w_pre"], t["w_post"], r_out=r, **how)
    assert got[0] is r and torch.equal(r, ro) and torch.equal(got[1], x)
    # a row's results do not depend on the rows beside it (without dropout, whose numbers go by position)
    full = ckl.add_norm(t["y"], t["r"], t["w_pre"], t["w_post"], gate=t["gate"])
    part = ckl.add_norm(t["y"][17:18], t["r"][17:18], t["w_pre"], t["w_post"], gate=t["gate"])
    assert torch.equal(full[1][17:18], part[1])


def test_an_input_given_twice(ckl):
    """The block's output as its own gate, and one weight in both places."""
    y, r, w = (torch.randn(*s, device="cuda:0") for s in ((7, 40), (7, 40), (40,)))
    for g in (y, r):
        a = ckl.add_norm(y, r, w, w, gate=g, stats=True)
        b = ckl.add_norm(y, r, w, w.clone(), gate=g.clone(), stats=True)
        assert all(torch.equal(u, v) for u, v in zip(a, b))
        ga = ckl.add_norm_bwd(y, r, w, w, a[2], y, r, gate=g)
        gb = ckl.add_norm_bwd(y, r, w, w.clone(), a[2], y.clone(), r.clone(), gate=g.clone())
        assert all(torch.equal(u, v) for u, v in zip(ga, gb)) and ga[4].shape == y.shape
    leaf = y.clone().requires_grad_()
    ro, x = ckl.residual_norm(leaf, r, w, gate=leaf, scale=0.5)
    ro.sum().backward()  # ro = r + y^2 / 2
    assert bool((leaf.grad - y).abs().max() <= 4 * 2.0 ** -24 * y.abs().max())  # two halves of y, each rounded once


def test_no_rows(ckl):
    e, w = torch.empty(0, 64, device="cuda:0"), torch.ones(64, device="cuda:0")
    ro, x, stats = ckl.add_norm(e, e, w, w, gate=w, stats=True)
    assert ro.shape == (0, 64) and stats.shape == (2, 0)
    dy, dr, dw_post, dw_pre, dgate = ckl.add_norm_bwd(e, e, w, w, stats, e, e, gate=w)
    assert dy.shape == (0, 64) and not dw_post.any() and not dw_pre.any() and not dgate.any()


def test_autograd(ckl):
    rng = np.random.default_rng(3)
    N, d = 21, 104
    leaves = [dev(rng.standard_normal(s), "f32").requires_grad_() for s in ((N, d), (N, d), (d,), (d,), (d,))]
    y, r, w_pre, w_post, gate = leaves
    ro, x = ckl.residual_norm(y.t().contiguous().t(), r, w_pre, w_post, gate, scale=0.5, p=0.2, seed=3, offset=1)
    a, b = torch.randn_like(ro), torch.randn_like(ro)
    ((ro * a).sum() + (x * b).sum()).backward()
    f = 0.5 * O.factors(N * d, 0.2, 3, 1).reshape(N, d)
    want = O.add_norm_grad(*(host(v.detach()) for v in leaves), f, float(np.float32(1e-6)), host(b), host(a))
    for t, name in zip(leaves, ("dy", "dr", "dw_pre", "dw_post", "dgate")):
        v, m = want[name]
        v, m = (v.sum(0), m.sum(0)) if t.dim() == 1 else (v, m)
        near(t.grad, v, m, N + 612, "f32", name)
    x2 = torch.randn(5, 33, device="cuda:0", requires_grad=True)
    ckl.dropout(x2, 0.4, 11, 2).sum().backward()
    assert torch.equal(x2.grad, ckl.drop(torch.ones_like(x2), 0.4, 11, 2))
    with torch.no_grad():
        assert not ckl.dropout(x2, 0.4, 11).requires_grad


def test_autograd_takes_the_offset_of_its_forward(ckl):
    at = torch.zeros(1, dtype=torch.int64, device="cuda:0")
    x = torch.randn(500, device="cuda:0", requires_grad=True)
    y = ckl.dropout(x, 0.5, 4, at)
    at += 1
    y.sum().backward()
    assert torch.equal(x.grad, ckl.drop(torch.ones_like(x), 0.5, 4, 0))


def test_captured_step_draws_anew(ckl):
    """A captured block end and its gradient, replayed with the offset moved on in the graph, with eager work between."""
    t, *_ = run(ckl, "bf16", 33, 256, True, True, "vector", 0.3, grads=())
    at = torch.zeros(1, dtype=torch.int64, device="cuda:0")
    dx = torch.randn(33, 256, device="cuda:0").to(torch.bfloat16)

    def step(offset):
        how = {"gate": t["gate"], "p": 0.3, "seed": 8, "offset": offset}
        ro, x, stats = ckl.add_norm(t["y"], t["r"], t["w_pre"], t["w_post"], stats=True, **how)
        return ro, x, *ckl.add_norm_bwd(t["y"], t["r"], t["w_pre"], t["w_post"], stats, dx, None, **how), ckl.drop(
            dx, 0.3, 8, offset)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(at)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(at)
        at.add_(1)
    at.zero_()
    for i in range(4):
        g.replay()
        torch.cuda.synchronize()
        assert int(at.item()) == i + 1
        want = step(i)
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_two_streams(ckl):
    t, ro, x, stats, g = run(ckl, "bf16", 2000, 1024, True, True, "vector", 0.1)
    how = {"gate": t["gate"], "scale": 0.7, "p": 0.1, "seed": 77, "offset": 5}
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(ckl.add_norm_bwd(t["y"], t["r"], t["w_pre"], t["w_post"], stats, t["dx"], t["dr"], **how))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, g))


def test_refusals(ckl):
    y, w = torch.randn(4, 64, device="cuda:0"), torch.ones(64, device="cuda:0")
    ok = ckl.add_norm(y, y, w, stats=True)
    for bad in ({"r": y[:3]}, {"r": y.half()}, {"w_pre": w[:8]}, {"w_post": w.bfloat16()}, {"gate": w[:8]},
                {"y": y.t().contiguous().t()}, {"y": y.cpu()}, {"eps": -1.0}, {"eps": float("nan")}, {"p": 1.5},
                {"p": float("nan")}, {"seed": -1}, {"seed": 1 << 64}, {"offset": -1}, {"offset": torch.zeros(1)},
                {"r_out": y.bfloat16()}, {"w_pre": None, "x_out": y}):
        with pytest.raises(ValueError):
            ckl.add_norm(**{"y": y, "r": y, "w_pre": w, **bad})
    with pytest.raises(ckl.CklError):
        ckl.add_norm(y[:, :60].contiguous(), y[:, :60].contiguous(), w[:60].contiguous())
    for bad in ({"stats": None}, {"stats": ok[2][:1]}, {"dx": None, "dr_out": None}, {"w_pre": None}, {"dx": y[:2]}):
        with pytest.raises(ValueError):
            ckl.add_norm_bwd(**{"y": y, "r": y, "w_pre": w, "w_post": None, "stats": ok[2], "dx": y, "dr_out": None, **bad})
    with pytest.raises(ValueError):
        ckl.drop(y.t(), 0.5, 1)
    with pytest.raises(ValueError):
        ckl.drop(y, 0.5, 1, out=y[:2])
    leaf = y.clone().requires_grad_()
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(g):
            ckl.dropout(leaf, 0.5, 1)
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(g):
            ckl.residual_norm(leaf, y, w)
