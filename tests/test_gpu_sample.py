"""Sampling on the GPU against the definition in extended precision.

Tokens have to be equal: masses and borders are held to about 1e-13 of a row's
total, so a token could only differ where a random border lies that close.  A
log-probability is rounded once to fp32 (2^-24 of its value) from masses good
to 1e-11.
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


def pick(v, r):
    return v[r].item() if torch.is_tensor(v) else v


def check(ckl, x, u, what="", **how):
    """Every row of x (a GPU tensor) against the oracle."""
    say(f"[case] sample {what} {tuple(x.shape)} {x.dtype} { {k: v if not torch.is_tensor(v) else 'per row' for k, v in how.items()} }")
    ids, logp = ckl.sample(x, u, **how)
    torch.cuda.synchronize()
    ids, logp, host, hu = ids.cpu().numpy(), logp.cpu().numpy(), x.float().cpu().numpy(), u.cpu().numpy()
    for r in range(x.shape[0]):
        i, lp = O.sample_row(host[r], hu[r], **{k: pick(v, r) for k, v in how.items()})
        assert ids[r] == i, (r, ids[r], i, hu[r])
        if i >= 0:
            assert abs(logp[r] - lp) <= 2.0 ** -24 * abs(lp) + 1e-11, (r, logp[r], lp)
        else:
            assert logp[r] == -np.inf
    return ids


def rows(N, V, dtype, std=3.0, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * V + N)
    return (torch.randn(N, V, generator=g) * std).to("cuda:0").to(DT[dtype])


def uniforms(N, seed=0):
    g = torch.Generator().manual_seed(seed + 977)
    u = torch.rand(N, generator=g)
    u[0] = 0.0
    u[N - 1] = 1 - 2.0 ** -24
    return u.to("cuda:0")


SETTINGS = [
    {}, {"temperature": 0.7}, {"temperature": 0.0}, {"top_k": 1}, {"top_k": 50}, {"top_k": 50, "top_p": 0.9},
    {"top_k": 512}, {"top_k": 513, "temperature": 1.3}, {"top_k": 3000, "top_p": 0.8}, {"top_p": 0.9}, {"top_p": 0.0},
    {"top_p": 0.5, "min_p": 0.02}, {"min_p": 0.05}, {"min_p": 1.0}, {"top_k": 40, "min_p": 0.1, "temperature": 2.0},
    {"top_k": 2000, "top_p": 0.95, "min_p": 0.001, "temperature": 1.5},
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 9, 100, 515, 5003, 32000])
def test_settings(ckl, dtype, V):
    for i, how in enumerate(SETTINGS):
        check(ckl, rows(9, V, dtype, seed=i), uniforms(9, i), **how)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_full_vocabulary(ckl, dtype):
    for i, how in enumerate(({}, {"top_p": 0.95}, {"top_k": 100, "top_p": 0.9}, {"top_k": 5000}, {"min_p": 0.01})):
        check(ckl, rows(5, 201088, dtype, seed=i), uniforms(5, i), **how)


@pytest.mark.parametrize("how", [{"temperature": t} for t in (1e-30, 1e-3, 0.05, 30.0, 1e30, float("inf"))]
                         + [{"temperature": 1e-3, "top_k": 900}, {"temperature": 30.0, "top_p": 0.7, "min_p": 0.9}])
def test_temperatures(ckl, how):
    check(ckl, rows(6, 4001, "f32"), uniforms(6), **how)
    check(ckl, rows(6, 4001, "bf16"), uniforms(6), **how)


def test_settings_per_row(ckl):
    N = 40
    g = torch.Generator().manual_seed(5)
    how = {"temperature": torch.rand(N, generator=g) * 2, "top_k": torch.randint(-3, 900, (N,), generator=g).to(torch.int32),
           "top_p": torch.rand(N, generator=g) * 1.3 - 0.1, "min_p": torch.rand(N, generator=g) * 0.2 - 0.05}
    how["temperature"][3], how["temperature"][4], how["temperature"][5] = 0.0, -1.0, float("nan")
    how["top_p"][6], how["min_p"][7], how["min_p"][8], how["top_k"][9] = float("nan"), float("nan"), 7.0, 1 << 30
    how = {k: v.to("cuda:0") for k, v in how.items()}
    for dtype in ("bf16", "f32"):
        check(ckl, rows(N, 6000, dtype), uniforms(N), **how)
    check(ckl, rows(N, 6000, "f32"), uniforms(N), temperature=how["temperature"])
    check(ckl, rows(N, 6000, "f32"), uniforms(N), top_k=how["top_k"], top_p=0.9)


@pytest.mark.parametrize("how", [{}, {"top_k": 7}, {"top_k": 600}, {"top_p": 0.5}, {"min_p": 0.1}])
def test_masks_infinities_and_nan(ckl, how):
    for dtype in ("bf16", "f32"):
        x = rows(10, 3001, dtype)
        inf = float("inf")
        x[0] = -inf                       # nothing left
        x[1, 5:] = -inf                   # five tokens
        x[2, :-1] = -inf                  # the last token alone
        x[3] = torch.finfo(DT[dtype]).min  # every token at the type's lowest value
        x[4, ::2] = torch.finfo(DT[dtype]).min
        x[5, 7] = x[5, 2999] = inf
        x[6, 100:200] = float("nan")
        x[7] = float("nan")
        x[8] = torch.finfo(DT[dtype]).max
        x[9, 1:] = -inf
        x[9, 0] = float("nan")
        ids = check(ckl, x, uniforms(10), **how)
        assert ids[0] == -1 and ids[7] == -1 and ids[9] == -1 and ids[2] == 3000 and ids[5] in (7, 2999)


@pytest.mark.parametrize("V", [2048, 2049, 9000, 70000])
@pytest.mark.parametrize("how", [{}, {"top_k": 3}, {"top_k": 2100}, {"top_p": 0.5}, {"top_k": 5000, "top_p": 0.25}, {"min_p": 0.5}])
def test_equal_logits(ckl, V, how):
    # more equal logits than fit on the chip: borders are counts, tokens ranks in id order
    for dtype in ("bf16", "f32"):
        u = torch.tensor([0.0, 0.25, 0.5, 0.7, 1 - 2.0 ** -24], device="cuda:0")
        x = torch.full((5, V), 1.5, device="cuda:0").to(DT[dtype])
        check(ckl, x, u, "all equal", **how)
        x[:, ::3] = 0.0
        x[:, 1::3] = -0.0
        check(ckl, x, u, "two values, signed zeros", **how)


@pytest.mark.parametrize("how", [{}, {"top_k": 4000}, {"top_p": 0.6}, {"top_k": 30000, "top_p": 0.9, "temperature": 0.8}])
def test_tiny_and_large_logits(ckl, how):
    # bf16 values the counted path leaves to the general one, or has to look at twice
    g = torch.Generator().manual_seed(9)
    u = uniforms(8)
    base = torch.randn(8, 5000, generator=g).to("cuda:0")
    for x in (base * 1e-9, base * 1e-9 * (base > 0), base * 200, base * 200 - 800, base * 3e37, -base.abs() * 1e3 - 300,
              torch.where(base > 1, base * 1e-10, base), torch.where(base > 1, torch.zeros_like(base), base)):
        check(ckl, x.to(torch.bfloat16), u, "tiny or large", **how)
        check(ckl, x.to(torch.bfloat16), u, "tiny or large", **dict(how, temperature=100.0))
    check(ckl, (base * 1e-9).to(torch.bfloat16), u, "tiny, resolved", **dict(how, temperature=1e-9))


@pytest.mark.parametrize("how", [{}, {"top_k": 4000}, {"top_p": 0.6}, {"top_k": 30000, "top_p": 0.9, "temperature": 0.8}])
def test_few_distinct_values(ckl, how):
    # one bin with far more tokens than fit, of several keys in it: narrowed by key digits
    g = torch.Generator().manual_seed(8)
    u = uniforms(8)
    x = torch.randint(0, 10, (8, 60000), generator=g).float().to("cuda:0")
    check(ckl, x.to(torch.bfloat16), u, "integers", **how)
    near = 1.0 + torch.randint(0, 300, (8, 60000), generator=g).float() * 2.0 ** -23
    check(ckl, near.to("cuda:0"), u, "neighbouring fp32 values", **how)
    check(ckl, (torch.rand(8, 60000, generator=g) * 1e-3).to("cuda:0"), u, "a narrow interval", **how)


@pytest.mark.parametrize("N,V", [(1, 32768), (1, 50001), (3, 201088), (7, 140000), (17, 100003), (64, 70000), (1, 1000003), (1, 1100000)])
def test_split_rows(ckl, N, V):
    # long rows of a small batch are counted by several workgroups; borders,
    # equal logits and the drawn one in any of the slices, also unaligned ones
    big = rows(N, V + 3, "bf16")
    for i, how in enumerate(({}, {"top_k": 40, "top_p": 0.9}, {"top_p": 0.8}, {"min_p": 0.02}, {"top_k": 3000})):
        check(ckl, big[:, i % 4: V + i % 4], uniforms(N, i), "split", **how)
    x = big[:, 1:V + 1]
    x[:] = float("-inf")
    x[:, V - 1] = 1.0
    x[:, V // 3] = 1.0
    assert set(check(ckl, x, uniforms(N), "two left").tolist()) <= {V // 3, V - 1}
    x[:] = 0.25
    check(ckl, x, uniforms(N), "all equal")
    x[0] = float("-inf")
    assert check(ckl, x, uniforms(N), "an empty row")[0] == -1


def test_without_a_workspace_the_same_bits(ckl):
    import ctypes

    from chunked_kl_loss_seq_amd import binding as B

    x, u = rows(2, 201088, "bf16"), uniforms(2)
    want = ckl.sample(x, u, top_p=0.9, temperature=0.7)
    how = B.Sampling(0.7, 0, 0.9, 0.0, None, None, None, None)
    ids, logp = torch.empty(2, dtype=torch.int32, device="cuda:0"), torch.empty(2, device="cuda:0")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert B.lib().ckl_sample(0, x.data_ptr(), 2, 201088, 201088, u.data_ptr(), ctypes.byref(how), ids.data_ptr(),
                              logp.data_ptr(), None, 0, stream) == 0
    assert torch.equal(ids, want[0]) and torch.equal(logp, want[1])
    assert B.lib().ckl_sample(0, x.data_ptr(), 2, 201088, 201088, u.data_ptr(), None, ids.data_ptr(), None, None, 0, stream) == 0
    assert torch.equal(ids, ckl.sample(x, u)[0])


def test_strided_and_unaligned_rows(ckl):
    for dtype in ("bf16", "f32"):
        big = rows(12, 5011, dtype)
        for view in (big[:, :5000], big[:, 1:5001], big[::3, 3:4000], big[:, 5:12], big[2:3, 1:], big.view(4, 3, 5011)[:, -1]):
            for how in ({}, {"top_k": 20}, {"top_p": 0.8}):
                check(ckl, view, uniforms(view.shape[0]), "strided", **how)
        one = rows(1, 700, dtype)
        check(ckl, one.expand(50, 700), uniforms(50), "one row many times")


def test_random_numbers_outside_their_range(ckl):
    u = torch.tensor([-1.0, float("nan"), 1.0, 5.0, float("inf")], device="cuda:0")
    for how in ({}, {"top_k": 10}):
        check(ckl, rows(5, 800, "f32"), u, **how)


def test_long_vocabulary(ckl):
    # 2^22 tokens: coarser integer masses
    check(ckl, rows(2, 1 << 22, "f32"), torch.tensor([0.3, 0.9], device="cuda:0"), top_p=0.9)
    check(ckl, rows(2, (1 << 22) + 3, "bf16"), torch.tensor([0.3, 0.9], device="cuda:0"))


def test_rows_beyond_32_bits(ckl):
    # rows whose offset passes 2^31 elements
    x = torch.empty(11000, 201088, dtype=torch.bfloat16, device="cuda:0")
    x[-1] = rows(1, 201088, "bf16")[0]
    check(ckl, x[10999:], uniforms(1), "alone")
    x[:-1] = 0
    u = torch.full((11000,), 0.37, device="cuda:0")
    ids, _ = ckl.sample(x, u, top_k=50)
    assert ids[-1].item() == O.sample_row(x[-1].float().cpu().numpy(), np.float32(0.37), top_k=50)[0]


def test_greedy_is_the_top_k_writers_first(ckl):
    x = rows(64, 30000, "bf16")
    first, _ = ckl.topk(x, 1)
    ids, logp = ckl.sample(x, uniforms(64), temperature=0)
    assert torch.equal(ids, first[:, 0]) and not logp.any()


def test_no_rows_and_outputs(ckl):
    x = rows(3, 50, "f32")
    ids, logp = ckl.sample(x[:0], uniforms(1)[:0])
    assert ids.shape == (0,) and logp.shape == (0,)
    i = torch.empty(3, dtype=torch.int32, device="cuda:0")
    p = torch.empty(3, device="cuda:0")
    got = ckl.sample(x, uniforms(3), ids_out=i, logp_out=p)
    assert got[0] is i and got[1] is p


def test_same_bits_every_time_and_on_two_streams(ckl):
    x = rows(300, 20000, "bf16")
    u = uniforms(300)
    want = [ckl.sample(x, u, **h) for h in ({}, {"top_k": 30}, {"top_p": 0.9})]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(4):
        with torch.cuda.stream(streams[turn % 2]):
            got = [ckl.sample(x, u, **h) for h in ({}, {"top_k": 30}, {"top_p": 0.9})]
        streams[turn % 2].synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("V", [1, 2, 3, 40, 5003])
def test_logits_about_zero(ckl, V):
    # every binary magnitude from 2^-30 to 2^-20 of either sign beside 0: where
    # the counts of bf16 values stop telling them apart
    g = torch.Generator().manual_seed(V)
    for N in (7, 80):
        e = torch.randint(-30, -19, (N, V), generator=g).double()
        x = torch.randint(-1, 2, (N, V), generator=g) * 2.0 ** e * (1 + torch.randint(0, 128, (N, V), generator=g) / 128)
        for r in range(0, N, 3):
            x[r] = x[r].abs().clamp(min=2.0 ** -30)  # no zero among them
        for how in ({}, {"temperature": 0.4}, {"top_p": 0.7}, {"top_k": 600, "min_p": 0.1}):
            check(ckl, x.float().to("cuda:0").bfloat16(), uniforms(N, V), **how)


@pytest.mark.parametrize("V", [5003, 24577, 30001, 100003, 262143, 262144])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_which_of_equal_logits(ckl, V, dtype):
    # n equal largest logits among ones that weigh nothing (e^-60 each): the
    # draw is the ceil(u n)-th of them in id order.  Rows start at every
    # alignment; the equal logits sit at the row's ends, at and beside the
    # borders of its thirds (in whole rounds of 8,192) and anywhere.
    N, ld = 72, V + 3
    rng = np.random.default_rng(V)
    b1 = V // 8 // 3 // 1024 * 8192
    marks = sorted({m + k for m in (0, b1, 2 * b1, V - 1) for k in range(-9, 10) if 0 <= m + k < V})
    x = np.full((N, ld), -40.0, np.float32)
    u, want = np.empty(N, np.float32), []
    for r in range(N):
        n = (1, 2, 5, 127, 128, 129, 300, 4000)[r % 8]
        if r % 3 == 0:
            at = rng.choice(marks, min(n, len(marks)), replace=False)
        elif r % 3 == 1:
            at = rng.choice(V, n, replace=False)
        else:  # one stretch
            at = rng.integers(0, V - n + 1) + np.arange(n)
        at = np.sort(at)
        k = int(rng.integers(len(at))) if r >= 16 else (0 if r < 8 else len(at) - 1)
        x[r, at] = 20.0
        u[r] = (k + 0.5) / len(at)
        want.append(int(at[k]))
    X = torch.from_numpy(x).to("cuda:0")
    X = (X.bfloat16() if dtype == "bf16" else X)[:, :V]
    ids, _ = ckl.sample(X, torch.from_numpy(u).to("cuda:0"))
    assert ids.tolist() == want


@pytest.mark.parametrize("seed", range(24))
def test_seeded_sweep(ckl, seed):
    # random sizes, row distances, distributions and settings, some per row
    g = torch.Generator().manual_seed(1000 + seed)

    def rand(lo, hi):
        return lo + (hi - lo) * torch.rand(1, generator=g).item()

    N = (1, 7, 66, 80)[seed % 4]
    V = int(2 ** rand(0, 16 if N < 60 else 14))
    x = torch.randn(N, V + seed % 5, generator=g) * rand(0.5, 8)
    shape = seed % 6
    if shape == 1:  # a grid of values
        x = (x * 2).round() / 2
    elif shape == 2:  # zeros of either sign
        x = torch.where(torch.rand(x.shape, generator=g) < 0.5, torch.zeros(()), x) * torch.sign(x)
    elif shape == 3:  # mostly masked
        x[torch.rand(x.shape, generator=g) < 0.95] = -float("inf")
    elif shape == 4:  # beyond +-256
        x *= 40
    elif shape == 5:  # tiny ones beside others
        x = torch.where(torch.rand(x.shape, generator=g) < 0.3, x * 1e-8, x * 0.01)
    how = {}
    for name, hi, as_type in (("temperature", 2.0, torch.float32), ("top_k", 900.0, torch.int32),
                              ("top_p", 1.0, torch.float32), ("min_p", 0.2, torch.float32)):
        turn = rand(0, 3)
        if turn < 1:
            how[name] = (torch.rand(N, generator=g) * hi).to(as_type).to("cuda:0")
        elif turn < 2:
            how[name] = int(rand(0, hi)) if as_type == torch.int32 else rand(0.05, hi)
    for dtype in ("bf16", "f32"):
        check(ckl, x.to("cuda:0").to(DT[dtype])[:, :V], uniforms(N, seed), **how)


def test_captured_and_replayed(ckl):
    x, u = rows(40, 9000, "bf16"), uniforms(40)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ckl.sample(x, u, top_k=20), ckl.sample(x, u, top_p=0.7)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = ckl.sample(x, u, top_k=20), ckl.sample(x, u, top_p=0.7)
    for turn in range(4):
        u.copy_(torch.roll(u, 3))
        x.copy_(torch.roll(x, 1, 0))
        g.replay()
        torch.cuda.synchronize()
        for got, how in ((a, {"top_k": 20}), (b, {"top_p": 0.7})):
            want = ckl.sample(x, u, **how)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals(ckl):
    from chunked_kl_loss_seq_amd import CklError

    x, u = rows(4, 100, "f32"), uniforms(4)
    for bad in (lambda: ckl.sample(x.half(), u), lambda: ckl.sample(x.cpu(), u), lambda: ckl.sample(x, u.cpu()),
                lambda: ckl.sample(x, u[:3]), lambda: ckl.sample(x, u.double()), lambda: ckl.sample(x[0], u),
                lambda: ckl.sample(x.t(), uniforms(100)), lambda: ckl.sample(x, u, top_k=torch.ones(4, device="cuda:0")),
                lambda: ckl.sample(x, u, temperature=torch.ones(3, device="cuda:0")),
                lambda: ckl.sample(x, u, ids_out=torch.zeros(4, device="cuda:0"))):
        with pytest.raises(ValueError):
            bad()
    for how in ({"temperature": -1.0}, {"temperature": float("nan")}, {"top_k": -1}, {"top_p": 1.5}, {"top_p": float("nan")},
                {"min_p": -0.1}, {"min_p": 2.0}):
        with pytest.raises(CklError):
            ckl.sample(x, u, **how)
