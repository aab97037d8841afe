"""What is dropped adds nothing to the residual, whatever the block's output holds, on the GPU: with w_post a NaN (or, at
eps = 0, a row of zeros) makes the whole row's u NaN, and drop(u) is 0 where an element goes."""
import pytest

from oracle import residual_oracle as O

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


def case(dtype, N, d, bad):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(d)
    y, r, w = (torch.randn(*s, device="cuda:0", generator=g).to(DT[dtype]) for s in ((N, d), (N, d), (d,)))
    if bad == "zeros":
        y[1] = 0
    else:
        y[1, d // 2] = float(bad)
    return y, r, w


# a row in lanes, in a wave by two vectors, in several waves, in more than 512 threads
@pytest.mark.parametrize("d", [24, 1000, 2880, 8200])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", ["nan", "zeros"])
@pytest.mark.parametrize("gated", [None, "vector", "full"])
def test_dropped_elements_keep_the_residual(ckl, d, dtype, bad, gated):
    N, p = 4, 0.4
    y, r, w = case(dtype, N, d, bad)
    gate = {None: None, "vector": w, "full": r}[gated]
    eps = 0.0 if bad == "zeros" else 1e-6
    kept = torch.from_numpy(O.factors(N * d, p, 7, 3).reshape(N, d) != 0).to("cuda:0")
    clean = ckl.add_norm(r, r, w, w, gate=gate, p=p, seed=7, offset=3, eps=eps)[0]
    ro, x, _ = ckl.add_norm(y, r, w, w, gate=gate, p=p, seed=7, offset=3, eps=eps)
    assert bool(ro[1][kept[1]].isnan().all())
    assert torch.equal(ro[1][~kept[1]], r[1][~kept[1]])
    assert bool(x[1].isnan().all()) and bool(ro[[0, 2, 3]].isfinite().all()) and bool(clean.isfinite().all())
    ro, x, _ = ckl.add_norm(y, r, None, w, gate=gate, p=p, seed=7, offset=3, eps=eps)
    assert x is None and torch.equal(ro[1][~kept[1]], r[1][~kept[1]])


@pytest.mark.parametrize("d", [24, 2880])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", ["nan", "inf", "zeros"])
def test_everything_dropped(ckl, d, dtype, bad):
    """p = 1: r passes through, and x is its norm, with finite gradients of r."""
    y, r, w = case(dtype, 3, d, bad)
    eps = 0.0 if bad == "zeros" else 1e-6
    ro, x, stats = ckl.add_norm(y, r, w, w, p=1.0, seed=7, offset=3, eps=eps, stats=True)
    want = ckl.add_norm(r, r, w, None, scale=0.0, eps=eps)  # the same without a branch
    assert torch.equal(ro, r) and torch.equal(x, want[1])
    dx = torch.ones_like(r)
    dr = ckl.add_norm_bwd(y, r, w, w, stats, dx, dx, p=1.0, seed=7, offset=3, eps=eps)[1]
    assert bool(dr.isfinite().all())


def test_infinity(ckl):
    """An infinite y: u is 0 beside it and NaN at it; where it goes, the row stays finite."""
    d, p = 64, 0.5
    kept = torch.from_numpy(O.factors(d, p, 7, 3) != 0).to("cuda:0")
    r, w = torch.randn(1, d, device="cuda:0"), torch.ones(d, device="cuda:0")
    for at, there in ((int(kept.nonzero()[0]), True), (int((~kept).nonzero()[0]), False)):
        y = torch.randn(1, d, device="cuda:0")
        y[0, at] = float("inf")
        ro, x, _ = ckl.add_norm(y, r, w, w, p=p, seed=7, offset=3)
        assert bool(ro[0, at].isnan()) == there and bool(x.isnan().any()) == there
        others = torch.arange(d, device="cuda:0") != at
        assert torch.equal(ro[0][others], r[0][others])


def test_a_whole_row_dropped_beside_kept_ones(ckl):
    """A row whose elements all go, where the lanes past its end, and the next row, keep theirs."""
    d, p = 24, 0.9
    for offset in range(2000):
        f = O.factors(3 * d, p, 7, offset).reshape(3, d)
        if not f[1].any() and f[2, :8].any():
            break
    assert not f[1].any() and f[2, :8].any()
    y, r, w = case("f32", 3, d, "nan")
    ro, x, stats = ckl.add_norm(y, r, w, w, p=p, seed=7, offset=offset, stats=True)
    assert torch.equal(ro[1], r[1]) and bool(x.isfinite().all())
    dr = ckl.add_norm_bwd(y, r, w, w, stats, torch.ones_like(r), torch.ones_like(r), p=p, seed=7, offset=offset)[1]
    assert bool(dr.isfinite().all())
