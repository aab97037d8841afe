"""Host-side checks of the vocabulary-end entry points: every bad argument returns
its status before any GPU work (the pointers are never dereferenced), so they
run without a GPU."""
import ctypes
import os

import pytest

from chunked_kl_loss_seq_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libckl.so not built")

EINVAL, EUNSUPPORTED, OK = -1, -5, 0
G = 1 << 20      # an aligned address that is never used
MIS = G + 2


def embed(dt=0, ids=G, W=G, scale=1.0, N=4, d=8, V=10, out=G):
    return B.lib().ckl_embed(dt, ids, W, scale, N, d, V, out, None)


@pytest.mark.parametrize("bad,want", [
    ({"dt": 2}, EINVAL), ({"N": -1}, EINVAL), ({"d": 0}, EINVAL), ({"V": 0}, EINVAL), ({"ids": None}, EINVAL),
    ({"W": None}, EINVAL), ({"out": None}, EINVAL), ({"W": G + 8}, EINVAL), ({"out": G + 8}, EINVAL),
    ({"ids": MIS}, EINVAL), ({"d": 12}, EUNSUPPORTED), ({"d": 1 << 21}, EUNSUPPORTED),
    ({"V": (1 << 26) + 1}, EUNSUPPORTED), ({"N": 1 << 26}, EUNSUPPORTED), ({"N": 0, "ids": None, "out": None}, OK),
])
def test_embed(bad, want):
    assert embed(**bad) == want


def workspace(N, d, V):
    b = ctypes.c_uint64(0)
    st = B.lib().ckl_embed_bwd_workspace(N, d, V, ctypes.byref(b))
    return st, b.value


def embed_bwd(dt=0, ids=G, dY=G, scale=1.0, N=4, d=8, V=10, acc=0, dW=G, ws=G, bytes_=1 << 30):
    return B.lib().ckl_embed_bwd(dt, ids, dY, scale, N, d, V, acc, dW, ws, bytes_, None)


@pytest.mark.parametrize("bad,want", [
    ({"dt": -1}, EINVAL), ({"ids": None}, EINVAL), ({"dY": None}, EINVAL), ({"dW": None}, EINVAL), ({"ws": None}, EINVAL),
    ({"dY": G + 8}, EINVAL), ({"dW": G + 4}, EINVAL), ({"ws": G + 128}, EINVAL), ({"bytes_": 0}, EINVAL),
    ({"bytes_": workspace(4, 8, 10)[1] - 1 if os.path.exists(B.LIB_PATH) else 0}, EINVAL), ({"d": 20}, EUNSUPPORTED),
    ({"N": 1 << 26}, EUNSUPPORTED), ({"N": (1 << 26) - 1, "d": 1 << 17, "bytes_": (1 << 63)}, EUNSUPPORTED),
    ({"N": 0, "acc": 1, "ids": None, "dY": None, "ws": None}, OK), ({"N": 0, "dW": None}, EINVAL),
])
def test_embed_bwd(bad, want):
    assert embed_bwd(**bad) == want


def test_embed_bwd_workspace():
    assert workspace(0, 8, 10) == (OK, 0)
    assert workspace(-1, 8, 10)[0] == EINVAL and workspace(4, 12, 10)[0] == EUNSUPPORTED
    assert B.lib().ckl_embed_bwd_workspace(4, 8, 10, None) == EINVAL
    last = 0
    for N in (1, 16, 17, 8192):
        st, b = workspace(N, 2880, 201088)
        assert st == OK and b % 256 == 0 and b >= last
        # keys, positions, a bit per token, two partial rows per tile of 16
        assert b >= 8 * N + 201088 // 8 + (-(-N // 16) * 2 * 2880 * 4 if N > 16 else 0)
        last = b
    # a long batch: two partial rows per 64 positions, no more than a fraction of dY
    assert workspace(262144, 2880, 201088)[1] < 262144 * 2880 * 2 // 4


def sample(dt=0, x=G, N=4, V=10, ld=10, u=G, ids=G, logp=G, work=None, bytes_=0, **how):
    s = B.Sampling(how.get("temperature", 1.0), how.get("top_k", 0), how.get("top_p", 1.0), how.get("min_p", 0.0),
                   how.get("Ts"), how.get("ks"), how.get("ps"), how.get("ms"))
    return B.lib().ckl_sample(dt, x, N, V, ld, u, ctypes.byref(s), ids, logp, work, bytes_, None)


@pytest.mark.parametrize("bad,want", [
    ({"dt": 3}, EINVAL), ({"x": None}, EINVAL), ({"u": None}, EINVAL), ({"ids": None}, EINVAL), ({"N": -1}, EINVAL),
    ({"V": 0}, EINVAL), ({"ld": -1}, EINVAL), ({"x": G + 1}, EINVAL), ({"dt": 1, "x": MIS}, EINVAL), ({"u": MIS}, EINVAL),
    ({"ids": MIS}, EINVAL), ({"logp": MIS}, EINVAL), ({"Ts": MIS}, EINVAL), ({"ks": MIS}, EINVAL),
    ({"temperature": -0.5}, EINVAL), ({"temperature": float("nan")}, EINVAL), ({"top_k": -1}, EINVAL),
    ({"top_p": 1.01}, EINVAL), ({"top_p": -0.01}, EINVAL), ({"top_p": float("nan")}, EINVAL), ({"min_p": 1.5}, EINVAL),
    ({"min_p": float("nan")}, EINVAL), ({"V": 200000, "work": G + 128, "bytes_": 1 << 30}, EINVAL),
    ({"V": 200000, "work": G, "bytes_": 100}, EINVAL), ({"V": (1 << 26) + 1}, EUNSUPPORTED), ({"N": 1 << 23}, EUNSUPPORTED),
    ({"N": 0, "x": None, "u": None, "ids": None, "logp": None}, OK),
])
def test_sample(bad, want):
    assert sample(**bad) == want


def test_sample_rows_fit_one_launch():
    # a workgroup of 1,024 threads per row, fewer than 2^32 threads a launch
    b = ctypes.c_uint64(0)
    assert sample(N=1 << 22) == EUNSUPPORTED
    assert B.lib().ckl_sample_workspace(0, 1 << 22, 10, ctypes.byref(b)) == EUNSUPPORTED
    assert B.lib().ckl_sample_workspace(0, (1 << 22) - 1, 10, ctypes.byref(b)) == OK


def test_sample_workspace():
    b = ctypes.c_uint64(7)
    f = B.lib().ckl_sample_workspace
    assert f(0, 0, 10, ctypes.byref(b)) == OK and b.value == 0
    assert f(0, 1, 201088, ctypes.byref(b)) == OK and 0 < b.value < 1 << 20
    for dt, N, V in ((0, 1, 30000), (0, 1000, 201088), (1, 1, 201088), (0, 1, 1 << 26)):  # rows not split
        assert f(dt, N, V, ctypes.byref(b)) == OK and b.value == 0
    assert f(2, 1, 10, ctypes.byref(b)) == EINVAL and f(0, 1, 10, None) == EINVAL and f(0, -1, 10, ctypes.byref(b)) == EINVAL
    assert f(0, 1, (1 << 26) + 1, ctypes.byref(b)) == EUNSUPPORTED


def quantize(dt=0, x=G, R=4, C=16, rows=1, q=G, s=G):
    return B.lib().ckl_quantize_fp8(dt, x, R, C, rows, q, s, None)


@pytest.mark.parametrize("bad,want", [
    ({"dt": 2}, EINVAL), ({"x": None}, EINVAL), ({"q": None}, EINVAL), ({"s": None}, EINVAL), ({"R": -1}, EINVAL),
    ({"C": 0}, EINVAL), ({"rows": 64}, EINVAL), ({"x": G + 8}, EINVAL), ({"q": G + 8}, EINVAL), ({"s": MIS}, EINVAL),
    ({"C": 24}, EUNSUPPORTED), ({"C": (1 << 20) + 16}, EUNSUPPORTED), ({"R": (1 << 26) + 1}, EUNSUPPORTED),
    ({"R": 1 << 26, "C": 1 << 16}, EUNSUPPORTED), ({"R": 0, "x": None, "q": None, "s": None}, OK),
])
def test_quantize(bad, want):
    assert quantize(**bad) == want


def matmul(dt=0, xq=G, xs=G, wq=G, ws=G, M=4, V=10, d=16, out=G):
    return B.lib().ckl_matmul_fp8(dt, xq, xs, wq, ws, M, V, d, out, None)


@pytest.mark.parametrize("bad,want", [
    ({"dt": 2}, EINVAL), ({"xq": None}, EINVAL), ({"xs": None}, EINVAL), ({"wq": None}, EINVAL), ({"ws": None}, EINVAL),
    ({"out": None}, EINVAL), ({"M": -1}, EINVAL), ({"V": 0}, EINVAL), ({"d": 0}, EINVAL), ({"xq": G + 8}, EINVAL),
    ({"wq": G + 8}, EINVAL), ({"xs": MIS}, EINVAL), ({"out": G + 1}, EINVAL), ({"dt": 1, "out": MIS}, EINVAL),
    ({"d": 24}, EUNSUPPORTED), ({"d": (1 << 20) + 16}, EUNSUPPORTED), ({"V": (1 << 26) + 1}, EUNSUPPORTED),
    ({"M": (1 << 26) + 1}, EUNSUPPORTED), ({"M": 1 << 20, "V": 1 << 20}, EUNSUPPORTED), ({"M": 0, "xq": None, "out": None}, OK),
])
def test_matmul(bad, want):
    assert matmul(**bad) == want
