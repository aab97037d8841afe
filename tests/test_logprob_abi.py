"""Host-side checks of the log-probabilities' entry points: every bad argument
returns its status before any GPU work (the pointers are never dereferenced), and
the planner is host code, so they run without a GPU."""
import ctypes
import os
import random

import pytest

from chunked_kl_loss_seq_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libckl.so not built")

EINVAL, EBUDGET, EUNSUPPORTED, OK = -1, -3, -5, 0
G = 1 << 20      # an aligned address that is never used
MIS = G + 2


def fwd(dt=0, x=G, N=4, V=100, ld=100, ids=G, T=2, mask=None, top=3, logp=G, ent=G, stats=G, tid=G, tlp=G, ws=None, n=0):
    return B.lib().ckl_logprobs(dt, x, N, V, ld, ids, T, mask, top, logp, ent, stats, tid, tlp, ws, n, None)


COMMON = [
    ({"dt": 2}, EINVAL), ({"N": -1}, EINVAL), ({"V": 0}, EINVAL), ({"ld": -1}, EINVAL), ({"T": -1}, EINVAL),
    ({"x": None}, EINVAL), ({"ids": None}, EINVAL), ({"x": G + 1}, EINVAL), ({"dt": 1, "x": MIS}, EINVAL),
    ({"ids": MIS}, EINVAL), ({"T": 2049}, EUNSUPPORTED), ({"V": (1 << 26) + 1}, EUNSUPPORTED),
    ({"N": 1 << 22}, EUNSUPPORTED),
]


@pytest.mark.parametrize("bad,want", COMMON + [
    ({"top": -1}, EINVAL), ({"top": 101}, EINVAL), ({"V": 1000, "top": 513}, EUNSUPPORTED), ({"logp": None}, EINVAL),
    ({"ent": None}, EINVAL), ({"stats": None}, EINVAL), ({"tid": None}, EINVAL), ({"tlp": None}, EINVAL),
    ({"logp": MIS}, EINVAL), ({"ent": MIS}, EINVAL), ({"stats": MIS}, EINVAL), ({"tid": MIS}, EINVAL), ({"tlp": MIS}, EINVAL),
    ({"V": 50000, "ws": G + 128, "n": 1 << 30}, EINVAL), ({"V": 50000, "ws": G, "n": 100}, EINVAL),
    ({"N": 0, "x": None, "ids": None, "logp": None, "ent": None, "stats": None}, OK),
])
def test_logprobs(bad, want):
    assert fwd(**bad) == want


def bwd(dt=0, x=G, N=4, V=100, ld=100, ids=G, T=2, mask=None, stats=G, ent=G, dlogp=G, dent=G, out=2 * G, ldo=100):
    return B.lib().ckl_logprobs_bwd(dt, x, N, V, ld, ids, T, mask, stats, ent, dlogp, dent, out, ldo, None)


@pytest.mark.parametrize("bad,want", COMMON + [
    ({"ldo": 99}, EINVAL), ({"stats": None}, EINVAL), ({"ent": None}, EINVAL), ({"dlogp": None}, EINVAL),
    ({"out": None}, EINVAL), ({"out": G + 1}, EINVAL), ({"stats": MIS}, EINVAL), ({"dlogp": MIS}, EINVAL),
    ({"dent": MIS}, EINVAL), ({"ent": MIS}, EINVAL), ({"out": G, "ld": 200}, EINVAL),
    ({"N": (1 << 22) - 1, "V": 40000, "ldo": 40000}, EUNSUPPORTED),
    ({"N": 0, "x": None, "ids": None, "stats": None, "out": None, "dlogp": None, "ent": None}, OK),
])
def test_logprobs_bwd(bad, want):
    assert bwd(**bad) == want


def test_logprobs_workspace():
    b = ctypes.c_uint64(7)
    f = B.lib().ckl_logprobs_workspace
    for N, V, top in ((0, 10, 0), (300, 201088, 20), (1, 8000, 5)):  # rows not split
        assert f(N, V, top, ctypes.byref(b)) == OK and b.value == 0
    for N, V, top in ((1, 201088, 20), (255, 1 << 26, 512), (61, 32000, 5), (1, 1 << 26, 0)):
        assert f(N, V, top, ctypes.byref(b)) == OK and 0 < b.value < 1 << 24 and b.value % 256 == 0
    assert f(1, 10, 11, ctypes.byref(b)) == EINVAL and f(1, 10, -1, ctypes.byref(b)) == EINVAL and f(1, 10, 1, None) == EINVAL
    assert f(1, 1000, 513, ctypes.byref(b)) == EUNSUPPORTED and f(1 << 22, 10, 1, ctypes.byref(b)) == EUNSUPPORTED


def head(dt=0, H=G, W=G, ids=G, mask=None, N=4, d=64, V=100, T=1, chunk=0, logp=G, ent=G, stats=G, ws=G, n=1 << 40):
    return B.lib().ckl_head_logprobs(dt, H, W, ids, mask, N, d, V, T, chunk, logp, ent, stats, ws, n, None)


HEAD = [
    ({"dt": 2}, EINVAL), ({"N": -1}, EINVAL), ({"d": 0}, EINVAL), ({"V": 0}, EINVAL), ({"T": -1}, EINVAL),
    ({"chunk": -1}, EINVAL), ({"H": None}, EINVAL), ({"W": None}, EINVAL), ({"ids": None}, EINVAL), ({"logp": None}, EINVAL),
    ({"stats": None}, EINVAL), ({"ws": None}, EINVAL), ({"n": 100}, EINVAL), ({"H": G + 8}, EINVAL), ({"W": G + 8}, EINVAL),
    ({"ids": MIS}, EINVAL), ({"logp": MIS}, EINVAL), ({"ent": MIS}, EINVAL), ({"stats": MIS}, EINVAL), ({"ws": G + 128}, EINVAL),
    ({"d": 60}, EUNSUPPORTED), ({"d": (1 << 20) + 8}, EUNSUPPORTED), ({"V": (1 << 26) + 1}, EUNSUPPORTED),
    ({"N": (1 << 26) + 1}, EUNSUPPORTED), ({"T": 2049}, EUNSUPPORTED), ({"N": 1 << 20, "T": 65}, EUNSUPPORTED),
]


@pytest.mark.parametrize("bad,want", HEAD + [
    ({"ent": None}, EINVAL),
    ({"N": 0, "H": None, "W": None, "ids": None, "logp": None, "ent": None, "stats": None, "ws": None, "n": 0}, OK),
])
def test_head_logprobs(bad, want):
    assert head(**bad) == want


def head_bwd(dt=0, H=G, W=G, ids=G, mask=None, N=4, d=64, V=100, T=1, chunk=0, logp=G, ent=G, stats=G, dlogp=G, dent=G, dH=G,
             dwt=0, acc=0, dW=G, ws=G, n=1 << 40):
    return B.lib().ckl_head_logprobs_bwd(dt, H, W, ids, mask, N, d, V, T, chunk, logp, ent, stats, dlogp, dent, dH, dwt, acc,
                                         dW, ws, n, None)


@pytest.mark.parametrize("bad,want", HEAD + [
    ({"ent": None}, EINVAL), ({"dlogp": None}, EINVAL), ({"dH": None}, EINVAL), ({"dW": None}, EINVAL), ({"dwt": 3}, EINVAL),
    ({"dt": 1, "dwt": 0}, EINVAL), ({"acc": 1}, EINVAL), ({"acc": 2, "dwt": 1}, EINVAL), ({"dH": G + 8}, EINVAL),
    ({"dW": G + 8}, EINVAL), ({"dlogp": MIS}, EINVAL), ({"dent": MIS}, EINVAL), ({"N": 0, "dW": None}, EINVAL),
    ({"N": 0, "acc": 1, "dwt": 1, "H": None, "ws": None, "n": 0}, OK),
])
def test_head_logprobs_bwd(bad, want):
    assert head_bwd(**bad) == want


def plan(back, dt, dwt, N, d, V, chunk=0, budget=0):
    c, b = ctypes.c_int64(-1), ctypes.c_uint64(0)
    st = B.lib().ckl_head_logprobs_plan(back, dt, dwt, N, d, V, chunk, budget, ctypes.byref(c), ctypes.byref(b))
    return st, c.value, b.value


def test_plan_keeps_its_budget():
    rng = random.Random(3)
    for _ in range(400):
        back, dt = rng.randint(0, 1), rng.randint(0, 1)
        dwt = 1 if dt == 1 else rng.randint(0, 1)
        N, d, V = int(2 ** rng.uniform(0, 22)), 8 * int(2 ** rng.uniform(0, 10)), int(2 ** rng.uniform(0, 18))
        budget = int(2 ** rng.uniform(20, 36))
        st, c, b = plan(back, dt, dwt, N, d, V, 0, budget)
        assert st in (OK, EBUDGET)
        if st == OK:
            assert 1 <= c <= N and b <= budget and (c == N or c % 256 == 0)
            assert plan(back, dt, dwt, N, d, V, c, budget)[0] == OK
            es = 4 if dt else 2
            # at least a chunk's exp or gradient values, or its slices' statistics
            assert b >= (c * V * es if back else c * (-(-V // 128)) * 12)


def test_plan():
    assert plan(0, 0, 0, 0, 64, 100) == (OK, 0, 0)
    st, c, b = plan(1, 0, 0, 4096, 2880, 201088)
    assert st == OK and c == 4096 and b < 3 << 30
    # a bf16 dW over several chunks keeps its fp32 sums in the workspace
    assert plan(1, 0, 0, 4096, 2880, 201088, 2048)[2] - plan(1, 0, 1, 4096, 2880, 201088, 2048)[2] == 201088 * 2880 * 4
    assert plan(1, 0, 0, 1 << 20, 2880, 201088, 0, 1 << 20)[0] == EBUDGET
    assert plan(0, 0, 0, 1 << 22, 64, 100, (1 << 20) + 1)[0] == EUNSUPPORTED
    assert plan(2, 0, 0, 1, 8, 1)[0] == EINVAL and plan(1, 1, 0, 1, 8, 1)[0] == EINVAL
