"""Cases of the operators around the vocabulary table: the embedding lookup and its gradient, sampling from logits,
and the head's product with an 8-bit weight, each with its plain form and its value in 64 bits.

A case is one call as a program makes it: a decode step's lookup, sample and head product on one or a few rows, a
training step's lookup and gradient on a whole batch, and the teacher's logits of a chunk of positions.  Sizes are
those of the workloads (201,088 x 2,880, 128,256, 32,000 x 2,048 and 4,096 x 256 heads; 32,768 and 4,096 positions)
and odd ones beside them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0


def listed():
    return [
        # one token of a decode step, and a training batch of one 32K-token sequence whose tail is padding
        {"name": "embed-decode", "op": "embed", "N": 1, "V": 201088, "d": 2880, "dtype": "bf16", "pad": 0.0},
        {"name": "embed-train-32k", "op": "embed", "N": 32768, "V": 201088, "d": 2880, "dtype": "bf16", "pad": 0.1},
        # the gradient of a small fp32 model, of a 4,096-token batch, and of the 32K-token sequence
        {"name": "embed-bwd-tiny", "op": "embed_bwd", "N": 256, "V": 4096, "d": 256, "dtype": "f32", "pad": 0.0},
        {"name": "embed-bwd-4k", "op": "embed_bwd", "N": 4096, "V": 32000, "d": 2048, "dtype": "bf16", "pad": 0.05},
        {"name": "embed-bwd-32k", "op": "embed_bwd", "N": 32768, "V": 201088, "d": 2880, "dtype": "bf16", "pad": 0.0},
        # a decode step of one request, a serving batch with each request's own settings, restricted sampling of a
        # batch, and unrestricted sampling of positions (students trained on their own samples)
        {"name": "sample-decode", "op": "sample", "N": 1, "V": 201088, "dtype": "bf16", "temperature": 0.8,
         "top_k": 50, "top_p": 0.95, "min_p": 0.0, "per_row": False, "masked": 0},
        {"name": "sample-serving", "op": "sample", "N": 61, "V": 32000, "dtype": "f32", "temperature": 0.7,
         "top_k": 40, "top_p": 0.9, "min_p": 0.05, "per_row": True, "masked": 0},
        {"name": "sample-top-p", "op": "sample", "N": 512, "V": 128256, "dtype": "bf16", "temperature": 0.9,
         "top_k": 0, "top_p": 0.9, "min_p": 0.0, "per_row": False, "masked": 256},
        {"name": "sample-full", "op": "sample", "N": 1024, "V": 201088, "dtype": "bf16", "temperature": 1.0,
         "top_k": 0, "top_p": 1.0, "min_p": 0.0, "per_row": False, "masked": 0},
        # the 8-bit head: a decode step, a chunk of positions of the teacher's offline run, and an odd shape whose rows
        # are already in 8 bits
        {"name": "fp8-head-decode", "op": "fp8", "M": 1, "V": 201088, "d": 2880, "dtype": "bf16", "given": False},
        {"name": "fp8-head-chunk", "op": "fp8", "M": 2048, "V": 201088, "d": 2880, "dtype": "bf16", "given": False},
        {"name": "fp8-odd", "op": "fp8", "M": 333, "V": 32001, "d": 2064, "dtype": "f32", "given": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_bwd", "sample", "sample", "fp8", "fp8"])
    if op in ("embed", "embed_bwd"):
        d = 8 * _log_int(rng, 8, 500)
        N = _log_int(rng, 1, max(2, min(65536, 94000000 // d)))
        V = _log_int(rng, 500, 201088)
        return {"op": op, "N": N, "V": V, "d": d, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "pad": rng.choice([0.0, round(rng.uniform(0.0, 0.3), 3)])}
    if op == "sample":
        V = _log_int(rng, 200, 262144)
        N = _log_int(rng, 1, min(4096, 120000000 // V))
        return {"op": op, "N": N, "V": V, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "temperature": round(rng.uniform(0.3, 1.5), 3), "top_k": rng.choice([0, 0, _log_int(rng, 1, 2000)]),
                "top_p": rng.choice([1.0, round(rng.uniform(0.1, 0.99), 3)]),
                "min_p": rng.choice([0.0, 0.0, round(rng.uniform(0.005, 0.2), 3)]), "per_row": rng.random() < 0.4,
                "masked": rng.choice([0, 0, rng.randint(1, V // 2)])}
    d = 16 * _log_int(rng, 8, 256)
    V = _log_int(rng, 300, 201088)
    M = _log_int(rng, 1, max(2, min(8192, int(8e11 / (d * V)), int(4e8 / V))))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    return {"op": op, "M": M, "V": V, "d": d, "dtype": dtype, "given": dtype == "f32" or rng.random() < 0.4}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _tokens(g, N, V, pad):
    """Token ids of text: Zipf (exponent 1.1) over a shuffled vocabulary, and a padded tail of -1."""
    w = torch.arange(1, V + 1, device=DEV, dtype=torch.float64).pow_(-1.1)
    c = torch.cumsum(w, 0)
    r = torch.rand(N, generator=g, device=DEV, dtype=torch.float64) * c[-1]
    ids = torch.searchsorted(c, r).clamp_(max=V - 1)
    ids = torch.randperm(V, generator=g, device=DEV)[ids].to(torch.int32)
    cut = int(pad * N)
    if cut:
        ids[N - cut:] = -1
    return ids


def _blocks(x):
    """fp32 [R, C] padded with zeros to [R, ceil(C / 128), 128]."""
    R, C = x.shape
    n = -(-C // 128)
    return torch.nn.functional.pad(x, (0, 128 * n - C)).reshape(R, n, 128)


def _scale(amax):
    return torch.where(amax > 0, (amax / E4M3_MAX).clamp(min=2.0 ** -126), torch.ones_like(amax))


def _quantize_rows(x):
    """8-bit rows with a scale per 1 x 128 block: (e4m3 [R, C], fp32 [ceil(C / 128), R])."""
    b = _blocks(x.float())
    s = _scale(b.abs().amax(2))
    q = (b / s[:, :, None]).to(torch.float8_e4m3fn).reshape(x.shape[0], -1)[:, :x.shape[1]]
    return q.contiguous(), s.t().contiguous()


def _quantize_weight(w):
    """8-bit weight with a scale per 128 x 128 block: (e4m3 [V, C], fp32 [ceil(V / 128), ceil(C / 128)])."""
    V, C = w.shape
    rows = -(-V // 128)
    b = _blocks(torch.nn.functional.pad(w.float(), (0, 0, 0, 128 * rows - V))).reshape(rows, 128, -1, 128)
    s = _scale(b.abs().amax((1, 3)))
    q = (b / s[:, None, :, None]).to(torch.float8_e4m3fn).reshape(128 * rows, -1)[:V, :C]
    return q.contiguous(), s


def prepare(case, seed):
    g = _gen(seed)
    t = TYPES[case["dtype"]]
    if case["op"] in ("embed", "embed_bwd"):
        ids = _tokens(g, case["N"], case["V"], case["pad"])
        rows = case["V"] if case["op"] == "embed" else case["N"]
        x = torch.empty(rows, case["d"], device=DEV, dtype=t).normal_(0, 1.0, generator=g)
        return {"case": case, "ids": ids, "x": x, "scale": math.sqrt(case["d"])}
    if case["op"] == "sample":
        N, V = case["N"], case["V"]
        # a wide bulk and a few likely tokens a row, as a language model's logits are
        x = torch.empty(N, V, device=DEV, dtype=torch.float32).normal_(0, 2.0, generator=g)
        few = torch.randint(0, V, (N, 24), generator=g, device=DEV)
        up = 6.0 + 8.0 * torch.rand(N, 24, generator=g, device=DEV)
        x.scatter_reduce_(1, few, up, "amax")  # a token drawn twice keeps the larger value
        if case["masked"]:
            x[:, V - case["masked"]:] = -math.inf
        s = {"case": case, "x": x.to(t), "u": torch.rand(N, generator=g, device=DEV)}
        if case["per_row"]:
            r = torch.rand(4, N, generator=g, device=DEV)
            s["temperature"] = case["temperature"] * (0.5 + r[0])
            s["top_k"] = torch.where(r[1] < 0.3, torch.zeros_like(r[1]), 1 + r[1] * 2 * case["top_k"]).to(torch.int32)
            s["top_p"] = torch.where(r[2] < 0.3, torch.ones_like(r[2]), case["top_p"] * r[2])
            s["min_p"] = case["min_p"] * r[3]
        else:
            s.update({k: case[k] for k in ("temperature", "top_k", "top_p", "min_p")})
        return s
    M, V, d = case["M"], case["V"], case["d"]
    w = torch.empty(V, d, device=DEV, dtype=torch.float32).normal_(0, 0.02, generator=g)
    wq, ws = _quantize_weight(w)
    del w
    h = torch.empty(M, d, device=DEV, dtype=torch.float32).normal_(0, 1.0, generator=g)
    h *= torch.exp(torch.empty(d, device=DEV).normal_(0, 0.7, generator=g))  # some channels are large
    s = {"case": case, "wq": wq, "ws": ws}
    if case["given"]:
        s["xq"], s["xs"] = _quantize_rows(h)
    else:
        s["h"] = h.to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ one pass

def _plain_embed(s):
    V, ids = s["x"].shape[0], s["ids"].long()
    there = (ids >= 0) & (ids < V)
    rows = s["x"][ids.clamp(0, V - 1)].float() * s["scale"]
    return torch.where(there[:, None], rows, torch.zeros_like(rows)).to(s["x"].dtype)


def _plain_embed_bwd(s):
    V, ids = s["case"]["V"], s["ids"].long()
    there = (ids >= 0) & (ids < V)
    g = torch.where(there[:, None], s["x"].float(), torch.zeros((), device=DEV))
    dW = torch.zeros(V, s["x"].shape[1], device=DEV, dtype=torch.float32)
    return dW.index_add_(0, ids.clamp(0, V - 1), g).mul_(s["scale"])


def _column(v, n, dtype):
    return v.to(dtype)[:, None] if torch.is_tensor(v) else torch.full((n, 1), v, device=DEV, dtype=dtype)


def _plain_sample(s):
    """Sorted, cumulated and searched in 64 bits: a token changes where its border moves."""
    N, V = s["x"].shape
    top, ids = torch.sort(s["x"].float(), dim=1, descending=True, stable=True)
    e = torch.exp((top.double() - top[:, :1].double()) / _column(s["temperature"], N, torch.float64))
    c = torch.cumsum(e, 1)
    k = _column(s["top_k"], N, torch.int64)
    k = torch.where((k <= 0) | (k > V), V, k)
    mass = c.gather(1, k - 1)
    p = _column(s["top_p"], N, torch.float64)
    reach = (c < p * mass).sum(1, keepdim=True).clamp(max=V - 1)
    mass = torch.where(p < 1, torch.minimum(mass, c.gather(1, reach)), mass)
    likely = (e >= _column(s["min_p"], N, torch.float64)).sum(1, keepdim=True)
    mass = torch.minimum(mass, c.gather(1, (likely - 1).clamp(min=0)))
    j = (c <= s["u"].double()[:, None] * mass).sum(1, keepdim=True).clamp(max=V - 1)
    logp = torch.log(e.gather(1, j) / mass)
    return ids.gather(1, j)[:, 0].to(torch.int32), logp[:, 0].float()


def _plain_fp8(s):
    xq, xs = (s["xq"], s["xs"]) if s["case"]["given"] else _quantize_rows(s["h"])
    x = _blocks(xq.float()) * xs.t()[:, :, None]
    w = s["wq"].float()
    V, d = w.shape
    w = w * s["ws"].repeat_interleave(128, 0)[:V].repeat_interleave(128, 1)[:, :d]
    return (x.reshape(x.shape[0], -1)[:, :d] @ w.t()).to(TYPES[s["case"]["dtype"]])


def run(state):
    op = state["case"]["op"]
    if own:
        import chunked_kl_loss_seq_amd as ckl

        if op == "embed":
            return ckl.embed(state["ids"], state["x"], scale=state["scale"])
        if op == "embed_bwd":
            return ckl.embed_bwd(state["ids"], state["x"], state["case"]["V"], scale=state["scale"])
        if op == "sample":
            return ckl.sample(state["x"], state["u"], temperature=state["temperature"], top_k=state["top_k"],
                              top_p=state["top_p"], min_p=state["min_p"])
        out = TYPES[state["case"]["dtype"]]
        if state["case"]["given"]:
            return ckl.matmul_fp8(state["xq"], state["xs"], state["wq"], state["ws"], dtype=out)
        return ckl.logits_fp8(state["h"], state["wq"], state["ws"], dtype=out)
    return {"embed": _plain_embed, "embed_bwd": _plain_embed_bwd, "sample": _plain_sample, "fp8": _plain_fp8}[op](state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "embed":
        N, V, d = case["N"], case["V"], case["d"]
        return {"bytes": 4 * N + size * d * (min(N, V) + N), "flops": N * d}
    if case["op"] == "embed_bwd":
        N, V, d = case["N"], case["V"], case["d"]
        return {"bytes": 4 * N + size * N * d + 4 * V * d, "flops": N * d + V * d}
    if case["op"] == "sample":
        N, V = case["N"], case["V"]
        return {"bytes": size * N * V + 12 * N, "flops": 4 * N * V}
    M, V, d = case["M"], case["V"], case["d"]
    n = -(-d // 128)
    rows = (M * d + 4 * M * n) if case["given"] else 2 * M * d
    return {"bytes": V * d + 4 * -(-V // 128) * n + rows + size * M * V, "flops": 2 * M * V * d}


# ------------------------------------------------------------------ 64 bits

def _exact_embed(s):
    V, ids = s["x"].shape[0], s["ids"].long()
    out = torch.zeros(ids.numel(), s["x"].shape[1], device=DEV, dtype=torch.float64)
    at = torch.nonzero((ids >= 0) & (ids < V))[:, 0]
    out[at] = s["x"].index_select(0, ids[at]).double().mul_(float(np.float32(s["scale"])))
    return out


def _exact_embed_bwd(s):
    """Sums of runs of the sorted tokens, as differences of running sums."""
    V, d = s["case"]["V"], s["x"].shape[1]
    ids, order = torch.sort(s["ids"].long(), stable=True)
    order = order[(ids >= 0) & (ids < V)]
    ids = ids[(ids >= 0) & (ids < V)]
    out = torch.zeros(V, d, device=DEV, dtype=torch.float64)
    token, count = torch.unique_consecutive(ids, return_counts=True)
    end = torch.cumsum(count, 0)
    for at in range(0, d, 512):
        c = torch.cumsum(s["x"][order, at:at + 512].double(), 0)
        c = torch.cat([torch.zeros_like(c[:1]), c])
        out[token, at:at + 512] = c[end] - c[end - count]
    return out.mul_(float(np.float32(s["scale"])))


def _exact_sample(s):
    """Row by row: the ranking, then the shortest of the three prefixes, then the walk along its probabilities."""
    x, u = s["x"].double(), s["u"].double().tolist()
    N, V = x.shape
    one = {k: s[k].tolist() if torch.is_tensor(s[k]) else [s[k]] * N for k in ("temperature", "top_k", "top_p", "min_p")}
    tokens, logps = [], []
    for r in range(N):
        rank = torch.argsort(-x[r], stable=True)
        z = x[r][rank] / one["temperature"][r]
        w = (z - z[0]).exp()
        keep = int(one["top_k"][r]) if 0 < one["top_k"][r] < V else V
        prob = w[:keep] / w[:keep].sum()
        if one["top_p"][r] < 1:
            keep = min(keep, int(torch.searchsorted(torch.cumsum(prob, 0), one["top_p"][r])) + 1)
        keep = max(1, min(keep, int((w >= one["min_p"][r]).sum())))
        prob = w[:keep] / w[:keep].sum()
        j = torch.searchsorted(torch.cumsum(prob, 0), u[r], right=True).clamp(max=keep - 1)
        tokens.append(rank[j])
        logps.append(prob[j].log())
    return torch.stack(tokens).to(torch.int32), torch.stack(logps)


def _e4m3(x):
    """The e4m3 value nearest to x (|x| <= 464), ties to even, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_fp8(s):
    d, V = s["wq"].shape[1], s["wq"].shape[0]
    n = -(-d // 128)
    if s["case"]["given"]:
        x = torch.cat([s["xq"][:, 128 * b:128 * b + 128].double() * s["xs"][b].double()[:, None] for b in range(n)], 1)
    else:
        parts = []
        for b in range(n):
            h = s["h"][:, 128 * b:128 * b + 128].double()
            a = h.abs().amax(1, keepdim=True)
            scale = torch.where(a > 0, (a / E4M3_MAX).float().double(), torch.ones_like(a))  # scales are held in fp32
            parts.append(_e4m3(h / scale) * scale)
        x = torch.cat(parts, 1)
    out = torch.empty(x.shape[0], V, device=DEV, dtype=torch.float64)
    for v in range(0, V, 16384):
        w = s["wq"][v:v + 16384].double()
        for b in range(n):
            rows = s["ws"][v // 128:v // 128 + 128, b].double().repeat_interleave(128)[:w.shape[0]]
            w[:, 128 * b:128 * b + 128] *= rows[:, None]
        out[:, v:v + 16384] = x @ w.t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "embed_bwd": _exact_embed_bwd, "sample": _exact_sample, "fp8": _exact_fp8}[case["op"]](s)
