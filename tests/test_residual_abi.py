"""Host-side checks of the residual's entry points: every bad argument returns its
status before any GPU work (the pointers are never dereferenced), so they run
without a GPU."""
import ctypes
import os

import pytest

from chunked_kl_loss_seq_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libckl.so not built")

EINVAL, EUNSUPPORTED, OK = -1, -5, 0
G = 1 << 20      # an aligned address that is never used
NAN = float("nan")


def dropout(dt=0, x=G, n=8, p=0.5, at=None, out=G, how=True):
    d = B.Drop(p, 1, 2, at)
    return B.lib().ckl_dropout(dt, x, n, ctypes.byref(d) if how else None, out, None)


@pytest.mark.parametrize("bad,want", [
    ({"dt": 2}, EINVAL), ({"n": -1}, EINVAL), ({"x": None}, EINVAL), ({"out": None}, EINVAL), ({"how": False}, EINVAL),
    ({"p": -0.1}, EINVAL), ({"p": 1.01}, EINVAL), ({"p": NAN}, EINVAL), ({"at": G + 4}, EINVAL), ({"x": G + 1}, EINVAL),
    ({"dt": 1, "out": G + 2}, EINVAL), ({"n": 1 << 37}, EUNSUPPORTED), ({"n": (1 << 37) - 8191}, EUNSUPPORTED),
    ({"n": 0, "x": None, "out": None}, OK),
])
def test_dropout(bad, want):
    assert dropout(**bad) == want


def norm(w_post, w_pre, gate, rows, eps, p):
    d = B.Drop(p, 1, 2, None) if p is not None else None
    return B.Norm(w_post, w_pre, gate, rows, 1.0, eps, ctypes.pointer(d) if d else None)


def add_norm(dt=0, y=G, r=G, N=4, d=64, w_post=G, w_pre=G, gate=G, rows=0, eps=1e-6, p=None, ro=G, x=2 * G, stats=G,
             how=True):
    h = norm(w_post, w_pre, gate, rows, eps, p)
    return B.lib().ckl_add_norm(dt, y, r, ctypes.byref(h) if how else None, N, d, ro, x, stats, None)


COMMON = [
    ({"dt": 7}, EINVAL), ({"y": None}, EINVAL), ({"r": None}, EINVAL), ({"N": -1}, EINVAL), ({"d": 0}, EINVAL),
    ({"how": False}, EINVAL), ({"rows": 2}, EINVAL), ({"eps": -1e-9}, EINVAL), ({"eps": NAN}, EINVAL), ({"p": 2.0}, EINVAL),
    ({"y": G + 1}, EINVAL), ({"w_post": G + 1}, EINVAL), ({"w_pre": G + 1}, EINVAL), ({"gate": G + 1}, EINVAL),
    ({"dt": 1, "r": G + 2}, EINVAL), ({"stats": G + 2}, EINVAL), ({"d": 60}, EUNSUPPORTED), ({"d": 16392}, EUNSUPPORTED),
    ({"N": (1 << 31) + 1}, EUNSUPPORTED),
]


@pytest.mark.parametrize("bad,want", COMMON + [
    ({"ro": None}, EINVAL), ({"x": None}, EINVAL), ({"w_pre": None}, EINVAL), ({"ro": G + 1}, EINVAL), ({"x": G + 1}, EINVAL),
    ({"x": G}, EINVAL), ({"N": 0, "y": None, "r": None, "ro": None, "x": None}, OK),
])
def test_add_norm(bad, want):
    assert add_norm(**bad) == want


def bwd(dt=0, y=G, r=G, N=4, d=64, w_post=G, w_pre=G, gate=G, rows=0, eps=1e-6, p=None, stats=G, dx=G, dr_in=G, dy=2 * G,
        dr=3 * G, dw_post=G, dw_pre=G, dgate=4 * G, ws=G, bytes_=1 << 30, how=True):
    h = norm(w_post, w_pre, gate, rows, eps, p)
    return B.lib().ckl_add_norm_bwd(dt, y, r, ctypes.byref(h) if how else None, N, d, stats, dx, dr_in, dy, dr, dw_post,
                                    dw_pre, dgate, ws, bytes_, None)


@pytest.mark.parametrize("bad,want", COMMON + [
    ({"stats": None}, EINVAL), ({"dx": None, "dr_in": None}, EINVAL), ({"w_pre": None, "dw_pre": None}, EINVAL),
    ({"dy": None}, EINVAL), ({"dr": None}, EINVAL), ({"dw_post": None}, EINVAL), ({"dw_pre": None}, EINVAL),
    ({"dgate": None}, EINVAL), ({"gate": None}, EINVAL), ({"ws": None}, EINVAL), ({"ws": G + 128}, EINVAL),
    ({"bytes_": 3 * 64 * 4 - 1}, EINVAL), ({"dx": G + 1}, EINVAL), ({"dr_in": G + 1}, EINVAL), ({"dy": G + 1}, EINVAL),
    ({"dr": G + 1}, EINVAL), ({"dw_post": G + 2}, EINVAL), ({"dw_pre": G + 2}, EINVAL), ({"dgate": G + 2}, EINVAL),
    ({"dy": 3 * G}, EINVAL), ({"dgate": 2 * G}, EINVAL), ({"rows": 1, "dgate": 3 * G}, EINVAL),
])
def test_add_norm_bwd(bad, want):
    assert bwd(**bad) == want


def test_workspace():
    b = ctypes.c_uint64(0)
    f = B.lib().ckl_add_norm_bwd_workspace
    assert f(0, 64, 3, ctypes.byref(b)) == OK and b.value == 0
    assert f(5, 64, 0, ctypes.byref(b)) == OK and b.value == 0
    for N, d in ((1, 8), (1000, 24), (40000, 2880), (1 << 31, 16384)):
        assert f(N, d, 3, ctypes.byref(b)) == OK and b.value % 256 == 0 and 12 * d <= b.value <= 2048 * 12 * 16384
    assert f(4, 64, 4, ctypes.byref(b)) == EINVAL and f(4, 64, -1, ctypes.byref(b)) == EINVAL
    assert f(4, 64, 1, None) == EINVAL and f(-1, 64, 1, ctypes.byref(b)) == EINVAL
    assert f(4, 60, 1, ctypes.byref(b)) == EUNSUPPORTED and f(4, 16392, 1, ctypes.byref(b)) == EUNSUPPORTED
