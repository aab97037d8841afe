"""Cases of the operators next to the head's loss: log-probabilities of given tokens with entropy and alternatives,
from logits and from hidden states; the residual's norms around a block; dropout whose mask is never stored.  Each
with its plain form and its value in 64 bits.

A case is one call as a program makes it, or a training step's call and its gradient: a decode step's report of the
token it took, the scores of positions under cached ids, a policy's log-probabilities with their gradient, a block's
end in a training step.  Sizes are those of the workloads (201,088 x 2,880, 128,256, 32,000 and 4,096 x 256 heads;
32,768 and 4,096 positions) and odd ones beside them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # a decode step's report: the token taken, the entropy and twenty alternatives of one row
        {"name": "logprobs-decode", "op": "logprobs", "N": 1, "V": 201088, "dtype": "bf16", "T": 1, "top": 20,
         "pad": 0, "banned": 0, "masked": 0.0, "grad": False},
        # a serving batch in fp32 whose rows end in the padding of the vocabulary, some tokens banned
        {"name": "logprobs-serving", "op": "logprobs", "N": 61, "V": 32000, "dtype": "f32", "T": 1, "top": 5,
         "pad": 64, "banned": 300, "masked": 0.0, "grad": False},
        # positions scored under a hundred cached ids each
        {"name": "logprobs-cached", "op": "logprobs", "N": 1024, "V": 201088, "dtype": "bf16", "T": 100, "top": 0,
         "pad": 0, "banned": 0, "masked": 0.0, "grad": False},
        # a policy's step on a model's logits: log-probabilities and entropy, and the logits' gradient
        {"name": "logprobs-train", "op": "logprobs", "N": 2048, "V": 128256, "dtype": "bf16", "T": 1, "top": 0,
         "pad": 0, "banned": 0, "masked": 0.1, "grad": True},
        # the same from hidden states: one token, a small fp32 model's step, and a step on 4,096 positions
        {"name": "head-decode", "op": "head", "N": 1, "V": 201088, "d": 2880, "dtype": "bf16", "T": 1, "masked": 0.0,
         "grad": False},
        {"name": "head-train-tiny", "op": "head", "N": 256, "V": 4096, "d": 256, "dtype": "f32", "T": 1, "masked": 0.0,
         "grad": True},
        {"name": "head-train-4k", "op": "head", "N": 4096, "V": 201088, "d": 2880, "dtype": "bf16", "T": 1,
         "masked": 0.1, "grad": True},
        # the end of a block for one token, for a training batch with its gradient, and for odd sizes in fp32
        {"name": "norm-decode", "op": "norm", "N": 1, "d": 2880, "dtype": "bf16", "post": True, "gate": "vector",
         "p": 0.0, "grad": False},
        {"name": "norm-train-32k", "op": "norm", "N": 32768, "d": 2880, "dtype": "bf16", "post": True,
         "gate": "vector", "p": 0.1, "grad": True},
        {"name": "norm-odd", "op": "norm", "N": 4099, "d": 1000, "dtype": "f32", "post": False, "gate": "full",
         "p": 0.0, "grad": True},
        # dropout of a small fp32 activation, and of a training batch; forward and gradient
        {"name": "dropout-small", "op": "dropout", "n": 65537, "dtype": "f32", "p": 0.2},
        {"name": "dropout-32k", "op": "dropout", "n": 94371840, "dtype": "bf16", "p": 0.1},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs", "head", "head", "norm", "norm", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "dropout":
        return {"op": op, "n": _log_int(rng, 1, 94371840), "dtype": dtype, "p": round(rng.uniform(0.0, 0.6), 3)}
    if op == "norm":
        d = 8 * _log_int(rng, 2, 1024)
        return {"op": op, "N": _log_int(rng, 1, min(65536, 94000000 // d)), "d": d, "dtype": dtype,
                "post": rng.random() < 0.6, "gate": rng.choice(["none", "vector", "full"]),
                "p": rng.choice([0.0, 0.0, round(rng.uniform(0.02, 0.4), 3)]), "grad": rng.random() < 0.6}
    if op == "logprobs":
        V = _log_int(rng, 100, 262144)
        N = _log_int(rng, 1, min(8192, 200000000 // V))
        grad = rng.random() < 0.4
        return {"op": op, "N": N, "V": V, "dtype": dtype, "T": rng.choice([0, 1, 1, _log_int(rng, 2, 200)]),
                "top": 0 if grad else rng.choice([0, 1, _log_int(rng, 2, min(V, 100))]),
                "pad": rng.choice([0, 0, rng.randint(1, 64)]), "banned": rng.choice([0, 0, rng.randint(1, V // 4)]),
                "masked": rng.choice([0.0, 0.0, round(rng.uniform(0.0, 0.5), 3)]), "grad": grad}
    d = 8 * _log_int(rng, 8, 500)
    V = _log_int(rng, 300, 201088)
    N = _log_int(rng, 1, min(8192, 400000000 // V, 2 * 10 ** 12 // (V * d)))
    return {"op": op, "N": N, "V": V, "d": d, "dtype": dtype, "T": rng.choice([1, 1, _log_int(rng, 2, 64)]),
            "masked": rng.choice([0.0, 0.0, round(rng.uniform(0.0, 0.5), 3)]), "grad": rng.random() < 0.6}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return torch.empty(*shape, device=DEV, dtype=dtype).normal_(0, std, generator=g)


def _upstream(g, s, N, T):
    """Per-token weights of either sign and the entropy's, of a mean over the batch."""
    s["dlogp"] = _normal(g, N, T) / N if T else None
    s["dentropy"] = (0.5 + torch.rand(N, generator=g, device=DEV)) * (0.1 / N)


def _mask(g, case):
    if not case["masked"]:
        return None
    return (torch.rand(case["N"], generator=g, device=DEV) >= case["masked"]).to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    t = TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "dropout":
        s["x"], s["dy"] = _normal(g, case["n"]).to(t), _normal(g, case["n"]).to(t)
        s["seed"], s["offset"] = 0x9E3779B97F4A7C15 * (seed + 1) % 2 ** 64, seed % 1000
        return s
    if case["op"] == "norm":
        N, d = case["N"], case["d"]
        # a block's output, and a residual that has grown over the layers, some of its channels large
        s["y"] = _normal(g, N, d).to(t)
        s["r"] = (_normal(g, N, d, std=3.0) * torch.exp(_normal(g, d, std=0.5))).to(t)
        s["w_post"] = (1.0 + _normal(g, d, std=0.2)).to(t) if case["post"] else None
        s["w_pre"] = (1.0 + _normal(g, d, std=0.2)).to(t)
        s["gate"] = {"none": lambda: None, "vector": lambda: _normal(g, d, std=0.5).to(t),
                     "full": lambda: torch.rand(N, d, generator=g, device=DEV).to(t)}[case["gate"]]()
        s["scale"], s["seed"], s["offset"] = 0.7, 0x9E3779B97F4A7C15 * (seed + 1) % 2 ** 64, seed % 1000
        if case["grad"]:
            s["dx"], s["dr"] = _normal(g, N, d).to(t), _normal(g, N, d, std=0.3).to(t)
        return s
    N, V, T = case["N"], case["V"], case["T"]
    s["ids"] = None
    if T:
        s["ids"] = torch.randint(0, V, (N, T), generator=g, device=DEV).to(torch.int32)
        # a few entries without a token, as the tail of a short list
        s["ids"][torch.rand(N, T, generator=g, device=DEV) < 0.02] = -1
    s["mask"] = _mask(g, case)
    if case["op"] == "logprobs":
        # a wide bulk and a few likely tokens a row, as a language model's logits are
        x = torch.zeros(N, V + case["pad"], device=DEV, dtype=t)
        x.normal_(0, 2.0, generator=g)
        few = torch.randint(0, V, (N, 24), generator=g, device=DEV)
        up = 6.0 + 8.0 * torch.rand(N, 24, generator=g, device=DEV)
        x.scatter_reduce_(1, few, up.to(t), "amax")
        x = x[:, :V]
        if case["banned"]:
            x.index_fill_(1, torch.randperm(V, generator=g, device=DEV)[:case["banned"]], -math.inf)
        if T:  # likely tokens among the given ones, never a banned one (its log-probability would be no number)
            some = few[:, torch.arange(T, device=DEV) % 24]
            likely = (torch.rand(N, T, generator=g, device=DEV) < 0.5) & (s["ids"] >= 0)
            s["ids"] = torch.where(likely, some.to(torch.int32), s["ids"])
            banned = torch.isinf(x.gather(1, s["ids"].long().clamp(min=0)))
            s["ids"] = torch.where(banned, torch.full_like(s["ids"], -1), s["ids"])
        s["x"] = x
    else:
        W = _normal(g, V, case["d"], std=0.02)
        s["H"] = _normal(g, N, case["d"])
        if T:  # the given token is likely
            c = 3.0 + 9.0 * torch.rand(N, 1, generator=g, device=DEV)
            s["H"] += c / (4e-4 * case["d"]) * W[s["ids"][:, 0].long().clamp(min=0)]
        s["H"], s["W"] = s["H"].to(t), W.to(t)
    if case["grad"]:
        _upstream(g, s, N, T)
    return s


# ------------------------------------------------------------------ one pass

M32 = 0xFFFFFFFF


def _philox(first, count, seed, offset):
    """Philox4x32-10 of the 64-bit counters first .. first + count - 1 in the low words, `offset` in the high ones:
    int64 [count, 4] of 32-bit words.  Products wrap in 64 bits, whose upper half is then the unsigned one."""
    i = torch.arange(first, first + count, device=DEV, dtype=torch.int64)
    c = [i & M32, i >> 32, torch.full_like(i, offset & M32), torch.full_like(i, offset >> 32)]
    k0, k1 = seed & M32, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & M32) ^ c[1] ^ k0, b & M32, ((a >> 32) & M32) ^ c[3] ^ k1, a & M32]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return torch.stack(c, 1)


def _kept(n, p, seed, offset):
    """Truth values [n] and the factor of what is kept: 16 bits an element, eight elements a counter."""
    border = min(65536, int(math.floor(p * 65536 + 0.5)))
    w = _philox(0, -(-n // 8), seed, offset)
    bits = torch.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n]
    return bits >= border, 65536.0 / max(1, 65536 - border)


def _plain_dropout(s):
    keep, f = _kept(s["case"]["n"], s["case"]["p"], s["seed"], s["offset"])
    zero = torch.zeros((), device=DEV)
    return tuple(torch.where(keep, s[k].float() * f, zero).to(s[k].dtype) for k in ("x", "dy"))


def _plain_norm(s):
    case, t = s["case"], s["y"].dtype
    y, r, w2 = s["y"].float(), s["r"].float(), s["w_pre"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    inv1 = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) if case["post"] else None
    w1 = s["w_post"].float() if case["post"] else None
    u = y * inv1 * w1 if case["post"] else y
    factor = torch.full((), s["scale"], device=DEV)
    if case["p"]:
        keep, f = _kept(y.numel(), case["p"], s["seed"], s["offset"])
        factor = torch.where(keep.view_as(y), factor * f, torch.zeros((), device=DEV))
    ro = r + factor * gate * u
    inv2 = torch.rsqrt((ro * ro).mean(1, keepdim=True) + EPS)
    n2 = ro * inv2
    out = (ro.to(t), (n2 * w2).to(t))
    if not case["grad"]:
        return out
    dx = s["dx"].float()
    a = dx * w2
    D = s["dr"].float() + inv2 * (a - n2 * (a * n2).mean(1, keepdim=True))
    dw2 = (dx * n2).sum(0)
    b = factor * D
    dgate = {"none": lambda: None, "vector": lambda: (b * u).sum(0), "full": lambda: (b * u).to(t)}[case["gate"]]()
    e = b * gate
    dw1 = None
    if case["post"]:
        n1 = y * inv1
        dw1 = (e * n1).sum(0)
        e = e * w1
        e = inv1 * (e - n1 * (e * n1).mean(1, keepdim=True))
    return [*out, *(v for v in (e.to(t), D.to(t), dw1, dw2, dgate) if v is not None)]


def _plain_logp(z, ids, mask, top):
    """(logp, entropy, (max, log of the sum)) of fp32 logits, and the ids and log-probabilities of the `top` largest."""
    N, V = z.shape
    m = z.amax(1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    logs = torch.log(total)
    entropy = (logs - (e * d.clamp(min=-1000.0)).sum(1, keepdim=True) / total)[:, 0]
    live = torch.ones(N, dtype=torch.bool, device=DEV) if mask is None else mask != 0
    zero = torch.zeros((), device=DEV)
    logp = None
    if ids is not None:
        logp = z.gather(1, ids.long().clamp(min=0)) - m - logs
        logp = torch.where((ids >= 0) & live[:, None], logp, zero)
    entropy = torch.where(live, entropy, zero)
    stats = torch.where(live, torch.cat([m, logs], 1).t(), zero)
    if not top:
        return logp, entropy, stats, None, None
    best, at = torch.sort(z, dim=1, descending=True, stable=True)
    best, at = best[:, :top], at[:, :top].to(torch.int32)
    there = live[:, None] & (best > -math.inf)
    return (logp, entropy, stats, torch.where(there, at, torch.full_like(at, -1)),
            torch.where(live[:, None], best - m - logs, zero))


def _plain_logits_grad(s, z, entropy, stats):
    """dlogp (onehot - p) - dentropy p (log p + entropy), of the rows that count."""
    l = z - stats[0][:, None] - stats[1][:, None]
    p = torch.exp(l)
    live = torch.ones(z.shape[0], device=DEV) if s["mask"] is None else s["mask"].float()
    given = torch.zeros(z.shape[0], device=DEV)
    if s["ids"] is not None:
        w = torch.where(s["ids"] >= 0, s["dlogp"], torch.zeros((), device=DEV)) * live[:, None]
        given = w.sum(1)
    G = -p * (given[:, None] + (s["dentropy"] * live)[:, None] * (l.clamp(min=-1000.0) + entropy[:, None]))
    if s["ids"] is not None:
        G.scatter_add_(1, s["ids"].long().clamp(min=0), w)
    return torch.where(live[:, None] != 0, G, torch.zeros((), device=DEV))


def _plain_logprobs(s):
    z = s["x"].float()
    out = _plain_logp(z, s["ids"], s["mask"], s["case"]["top"])
    got = [v for v in out if v is not None]
    if s["case"]["grad"]:
        got.append(_plain_logits_grad(s, z, out[1], out[2]).to(s["x"].dtype))
    return got


def _plain_head(s):
    H, W = s["H"].float(), s["W"].float()
    z = H @ W.t()
    logp, entropy, stats, _, _ = _plain_logp(z, s["ids"], s["mask"], 0)
    if not s["case"]["grad"]:
        return logp, entropy, stats
    G = _plain_logits_grad(s, z, entropy, stats)
    return logp, entropy, stats, (G @ W).to(s["H"].dtype), (G.t() @ H).to(s["W"].dtype)


def _own(s):
    import chunked_kl_loss_seq_amd as ckl

    case, op = s["case"], s["case"]["op"]
    if op == "dropout":
        return tuple(ckl.dropout(s[k], case["p"], s["seed"], s["offset"]) for k in ("x", "dy"))
    if op == "norm":
        how = {"gate": s["gate"], "scale": s["scale"], "p": case["p"], "seed": s["seed"], "offset": s["offset"], "eps": EPS}
        if not case["grad"]:
            return ckl.add_norm(s["y"], s["r"], s["w_pre"], s["w_post"], **how)[:2]
        ro, x, stats = ckl.add_norm(s["y"], s["r"], s["w_pre"], s["w_post"], stats=True, **how)
        grads = ckl.add_norm_bwd(s["y"], s["r"], s["w_pre"], s["w_post"], stats, s["dx"], s["dr"], **how)
        return [ro, x, *(v for v in grads if v is not None)]
    if op == "logprobs":
        out = ckl.logprobs(s["x"], s["ids"], top=case["top"], mask=s["mask"])
        got = [v for v in out if v is not None]
        if case["grad"]:
            got.append(ckl.logprobs_bwd(s["x"], s["ids"], out.entropy, out.stats, s["dlogp"], s["dentropy"],
                                        mask=s["mask"]))
        return got
    out = ckl.head_logprobs(s["H"], s["W"], s["ids"], mask=s["mask"])
    if not case["grad"]:
        return out.logp, out.entropy, out.stats
    dH, dW = ckl.head_logprobs_bwd(s["H"], s["W"], s["ids"], out.logp, out.entropy, out.stats, s["dlogp"],
                                   s["dentropy"], mask=s["mask"])
    return out.logp, out.entropy, out.stats, dH, dW


def run(state):
    if own:
        return _own(state)
    return {"dropout": _plain_dropout, "norm": _plain_norm, "logprobs": _plain_logprobs,
            "head": _plain_head}[state["case"]["op"]](state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "dropout":
        return {"bytes": 4 * size * case["n"], "flops": 2 * case["n"]}
    if case["op"] == "norm":
        n, d = case["N"] * case["d"], case["d"]
        full = n if case["gate"] == "full" else 0
        vectors = 1 + case["post"] + (case["gate"] == "vector")
        if not case["grad"]:
            return {"bytes": size * (4 * n + full + vectors * d), "flops": 8 * n}
        # forward 2 in, 2 out; gradient 4 in (the block's output, the residual, the two upstream ones), 2 out
        return {"bytes": size * (10 * n + 3 * full + vectors * d) + 4 * vectors * d, "flops": 24 * n}
    N, V, T = case["N"], case["V"], case["T"]
    live = N - int(case["masked"] * N)
    few = 8 * N * T + 12 * N
    if case["op"] == "logprobs":
        grad = size * (live + N) * V if case["grad"] else 0
        return {"bytes": size * live * V + grad + few + 8 * N * case["top"],
                "flops": (10 if case["grad"] else 4) * live * V}
    d = case["d"]
    one = 2 * live * V * d
    if not case["grad"]:
        return {"bytes": size * (V * d + live * d) + few, "flops": one}
    return {"bytes": 2 * size * (V * d + N * d) + few, "flops": 3 * one}


# ------------------------------------------------------------------ 64 bits

def _bits(n, seed, offset):
    """The 16-bit numbers of n elements, by the generator's definition in NumPy."""
    at = np.arange(-(-n // 8), dtype=np.uint64)
    low, sh = np.uint64(M32), np.uint64(32)
    x0, x1 = at & low, at >> sh
    x2, x3 = np.full_like(at, offset & M32), np.full_like(at, offset >> 32)
    key = [seed & M32, seed >> 32]
    for r in range(10):
        p, q = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        k = [np.uint64((key[0] + r * 0x9E3779B9) % 2 ** 32), np.uint64((key[1] + r * 0xBB67AE85) % 2 ** 32)]
        x0, x1, x2, x3 = (q >> sh) ^ x1 ^ k[0], q & low, (p >> sh) ^ x3 ^ k[1], p & low
    words = np.stack([x0, x1, x2, x3], 1).astype(np.uint32)
    return torch.from_numpy(words.view(np.uint16).reshape(-1)[:n].astype(np.int32)).to(DEV)


def _factors(n, p, s):
    """What dropout multiplies each of n elements with, in 64 bits."""
    cut = min(65536, math.floor(p * 65536 + 0.5))
    if cut == 65536:
        return torch.zeros(n, device=DEV, dtype=torch.float64)
    return (_bits(n, s["seed"], s["offset"]) >= cut).double() * (65536 / (65536 - cut))


def _exact_dropout(s):
    f = _factors(s["case"]["n"], s["case"]["p"], s)
    return s["x"].double() * f, s["dy"].double() * f


def _rms_grad(g, v):
    """The gradient at v of the rows v / sqrt(mean(v^2) + eps), under g."""
    q = (v * v).sum(1, keepdim=True) / v.shape[1] + EPS
    return g / q.sqrt() - v * (g * v).sum(1, keepdim=True) / (v.shape[1] * q ** 1.5)


def _exact_norm(s):
    case = s["case"]
    y, r = s["y"].double(), s["r"].double()
    f = float(np.float32(s["scale"])) * (_factors(y.numel(), case["p"], s).view_as(y) if case["p"] else torch.ones_like(y))
    if s["gate"] is not None:
        gate = s["gate"].double().expand_as(y)
    else:
        gate = torch.ones_like(y)
    unit = lambda v: v / ((v * v).sum(1, keepdim=True) / v.shape[1] + EPS).sqrt()  # noqa: E731
    n1 = unit(y) if case["post"] else y
    u = n1 * s["w_post"].double() if case["post"] else n1
    ro = r + f * gate * u
    n2 = unit(ro)
    out = [ro, n2 * s["w_pre"].double()]
    if not case["grad"]:
        return tuple(out)
    dx = s["dx"].double()
    D = s["dr"].double() + _rms_grad(dx * s["w_pre"].double(), ro)
    du = D * f * gate
    dy, dw1 = du, None
    if case["post"]:
        dw1 = (du * n1).sum(0)
        dy = _rms_grad(du * s["w_post"].double(), y)
    dg = D * f * u
    dgate = None if s["gate"] is None else dg.sum(0) if case["gate"] == "vector" else dg
    return [*out, *(v for v in (dy, D, dw1, (dx * n2).sum(0), dgate) if v is not None)]


def _exact_logp(z, s, top):
    logp = torch.log_softmax(z, 1)
    p = logp.exp()
    H = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    m = z.max(1).values
    stats = torch.stack([m, torch.logsumexp(z - m[:, None], 1)])
    off = torch.zeros_like(m, dtype=torch.bool) if s["mask"] is None else s["mask"] == 0
    got = [H.masked_fill(off, 0.0), stats.masked_fill(off, 0.0)]
    if s["ids"] is not None:
        none = (s["ids"] < 0) | off[:, None]
        got.insert(0, torch.gather(logp, 1, s["ids"].long().clamp(min=0)).masked_fill(none, 0.0))
    if top:
        at = torch.argsort(-z, dim=1, stable=True)[:, :top]
        v = torch.gather(logp, 1, at)
        at = torch.where((v == -math.inf) | off[:, None], torch.full_like(at, -1), at)
        got += [at.to(torch.int32), v.masked_fill(off[:, None], 0.0)]
    return got, logp, p, H, off


def _exact_grad(s, logp, p, H, off):
    up = s["dentropy"].double().masked_fill(off, 0.0)[:, None]
    G = -up * torch.where(p > 0, p * (logp + H[:, None]), torch.zeros_like(p))
    if s["ids"] is not None:
        w = s["dlogp"].double().masked_fill((s["ids"] < 0) | off[:, None], 0.0)
        G -= p * w.sum(1, keepdim=True)
        G.scatter_add_(1, s["ids"].long().clamp(min=0), w)
    return G


def _exact_logprobs(s):
    got, *rest = _exact_logp(s["x"].double(), s, s["case"]["top"])
    if s["case"]["grad"]:
        got.append(_exact_grad(s, *rest))
    return got


def _exact_head(s):
    H, W = s["H"].double(), s["W"].double()
    got, *rest = _exact_logp(H @ W.t(), s, 0)
    if s["case"]["grad"]:
        G = _exact_grad(s, *rest)
        got += [G @ W, G.t() @ H]
    return tuple(got)


def exact(case, seed):
    s = prepare(case, seed)
    return {"dropout": _exact_dropout, "norm": _exact_norm, "logprobs": _exact_logprobs,
            "head": _exact_head}[case["op"]](s)
