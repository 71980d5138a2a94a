"""Cases of the operators around a lookup of ragged sequences, for timing: the
dense embedding lookup and its gradient, layer norm in both directions, and
attention of each bag's queries over the bag's keys in both directions.

`own` picks what run() calls: the plain form in torch (False) or the library's
entry points (True).  exact() gives the same outputs from the definitions in
64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
PADDING = -1  # the padding token
EPS = 1e-5


# ------------------------------------------------------------------ cases
def _lookup(name, N, V, D, w, o, scale, zipf=0.9, pad=0.0):
    return {"name": name, "kind": "embed_lookup", "N": N, "V": V, "D": D, "w": w, "o": o, "scale": scale,
            "zipf": zipf, "pad": pad}


def _grad(name, N, V, D, g, o, scale, zipf=0.9, pad=0.0):
    return {"name": name, "kind": "embed_grad", "N": N, "V": V, "D": D, "g": g, "o": o, "scale": scale, "zipf": zipf,
            "pad": pad}


def _norm(name, kind, M, D, x, y, w):
    return {"name": name, "kind": kind, "M": M, "D": D, "x": x, "y": y, "w": w}


def _attend(name, kind, B, q, k, Hq, Hkv, D, t, masked=0.0):
    return {"name": name, "kind": kind, "B": B, "q_lo": q[0], "q_hi": q[1], "k_lo": k[0], "k_hi": k[1], "Hq": Hq,
            "Hkv": Hkv, "D": D, "t": t, "masked": masked}


def listed():
    return [
        # one serving step's tokens against a large vocabulary: latency
        _lookup("lookup-serve", 64, 131072, 1024, "bf16", "bf16", 32.0),
        # the long behaviour sequences' occurrences, fp32 weights read as 16-bit rows
        _lookup("lookup-longseq", 1500000, 1000000, 128, "fp32", "bf16", 1.0, pad=0.02),
        # a training batch's tokens, gradient of the whole weight
        _grad("grad-vocab", 65536, 131072, 512, "bf16", "fp32", 22.5, zipf=1.05),
        # the long behaviour sequences' gradient, hot tokens among them
        _grad("grad-longseq", 1500000, 1000000, 128, "bf16", "fp32", 1.0, pad=0.02),
        # the rows of one serving step
        _norm("norm-serve", "norm", 64, 256, "bf16", "bf16", "fp32"),
        # fp32 table rows of the long sequences narrowed to 16 bits, and their gradient
        _norm("norm-train-longseq", "norm_train", 1500000, 128, "fp32", "bf16", "fp32"),
        # wide activations of a training step
        _norm("norm-train-wide", "norm_train", 16384, 4096, "bf16", "bf16", "bf16"),
        # an odd width and a ragged row count
        _norm("norm-train-odd", "norm_train", 5003, 1001, "fp16", "fp16", "fp32"),
        # a handful of short bags: latency
        _attend("attend-small", "attend", 8, (1, 4), (0, 50), 4, 4, 32, "bf16"),
        # serving: one candidate against each user's long sequence, shared key heads
        _attend("attend-serve", "attend", 256, (1, 1), (1000, 5000), 8, 2, 128, "bf16"),
        # training: a few candidates for each user's long sequence, some keys masked
        _attend("attend-train-longseq", "attend_train", 256, (0, 16), (1000, 5000), 2, 2, 64, "fp16", masked=0.05),
        # training: many candidates over long sequences
        _attend("attend-train-ranking", "attend_train", 16, (512, 1024), (1024, 4096), 8, 4, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    kind = rng.choice(["embed_lookup", "embed_grad", "norm", "norm_train", "attend", "attend", "attend_train",
                       "attend_train"])
    types = ["fp32", "bf16", "fp16"]
    if kind.startswith("embed"):
        D = _log(rng, 8, 1024)
        if rng.random() < 0.7:
            D -= D % 8
        N = min(_log(rng, 1, 1500000), 190000000 // D)
        V = min(_log(rng, 100, 1000000), 128000000 // D)
        zipf, pad, scale = rng.uniform(0.5, 1.2), rng.choice([0.0, 0.05]), rng.choice([1.0, 0.5, math.sqrt(D)])
        a, b = rng.choice(types), rng.choice(types)
        c = _lookup("", N, V, D, a, b, scale, zipf, pad) if kind == "embed_lookup" else _grad("", N, V, D, a, b, scale,
                                                                                              zipf, pad)
    elif kind.startswith("norm"):
        D = _log(rng, 8, 8192)
        if rng.random() < 0.7:
            D -= D % 8
        c = _norm("", kind, min(_log(rng, 1, 1500000), 190000000 // D), D, rng.choice(types), rng.choice(types),
                  rng.choice(types))
    else:
        D = rng.choice([16, 24, 32, 40, 64, 64, 72, 96, 128, 128])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 1, 2, 3, 4])
        k_hi = _log(rng, 8, 5000)
        q_hi = rng.choice([1, _log(rng, 1, 16), _log(rng, 16, 1024)])
        # what the padded plain form holds: its scores and its keys
        most = min(536000000 // (Hkv * G * q_hi * k_hi), 330000000 // (Hkv * D * k_hi))
        B = max(1, min(_log(rng, 1, 512), most))
        k_lo = rng.choice([0 if B >= 8 else k_hi // 2, k_hi // 4, k_hi])
        c = _attend("", kind, B, (rng.choice([0, q_hi // 2, q_hi]), q_hi), (k_lo, k_hi), Hkv * G, Hkv, D,
                    rng.choice(["bf16", "fp16"]), rng.choice([0.0, 0.0, 0.1]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tokens(c, g):
    """Zipf-distributed tokens, hot ones scattered over the vocabulary; some padding."""
    p = torch.arange(1, c["V"] + 1, device="cuda", dtype=torch.float64).pow(-c["zipf"]).cumsum(0)
    u = torch.rand(c["N"], device="cuda", dtype=torch.float64, generator=g) * p[-1]
    rank = torch.searchsorted(p, u).clamp(max=c["V"] - 1)
    t = torch.randperm(c["V"], device="cuda", generator=g)[rank]
    if c["pad"]:
        t = torch.where(torch.rand(c["N"], device="cuda", generator=g) < c["pad"], PADDING, t)
    return t


def _rand(shape, dtype, g, mul=1.0, add=0.0):
    return torch.randn(shape, device="cuda", generator=g).mul_(mul).add_(add).to(DTYPES[dtype])


def _lengths(B, lo, hi):
    """B lengths spread evenly over [lo, hi]."""
    n = lo + np.rint((hi - lo) * np.arange(1, B + 1) / B).astype(np.int64)
    return np.minimum(n, hi)


def _offsets(B, lo, hi, rng):
    return np.concatenate([[0], np.cumsum(rng.permutation(_lengths(B, lo, hi)))]).astype(np.int64), hi


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["kind"] == "embed_lookup":
        s["weight"] = _rand((c["V"], c["D"]), c["w"], g, mul=1.0 / math.sqrt(c["D"]))
        s["tokens"] = _tokens(c, g)
    elif c["kind"] == "embed_grad":
        s["tokens"] = _tokens(c, g)
        s["grad"] = _rand((c["N"], c["D"]), c["g"], g)
    elif c["kind"].startswith("norm"):
        s["x"] = _rand((c["M"], c["D"]), c["x"], g, mul=1.5, add=0.25)
        s["weight"] = _rand((c["D"],), c["w"], g, mul=0.2, add=1.0)
        s["bias"] = _rand((c["D"],), c["w"], g, mul=0.2)
        if c["kind"] == "norm_train":
            s["grad"] = _rand((c["M"], c["D"]), c["y"], g)
    else:
        rng = np.random.default_rng([seed, 5])
        qo, s["max_q"] = _offsets(c["B"], c["q_lo"], c["q_hi"], rng)
        ko, s["max_k"] = _offsets(c["B"], c["k_lo"], c["k_hi"], rng)
        s["q_offsets"], s["k_offsets"] = torch.from_numpy(qo).cuda(), torch.from_numpy(ko).cuda()
        s["q"] = _rand((int(qo[-1]), c["Hq"], c["D"]), c["t"], g)
        s["k"] = _rand((int(ko[-1]), c["Hkv"], c["D"]), c["t"], g)
        s["v"] = _rand((int(ko[-1]), c["Hkv"], c["D"]), c["t"], g)
        s["mask"] = None
        if c["masked"]:
            s["mask"] = torch.rand(int(ko[-1]), device="cuda", generator=g) >= c["masked"]
        if c["kind"] == "attend_train":
            s["grad"] = _rand(tuple(s["q"].shape), c["t"], g)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["kind"] == "embed_lookup":
        return _plain_lookup(c, state)
    if c["kind"] == "embed_grad":
        return _plain_grad(c, state)
    if c["kind"].startswith("norm"):
        return _plain_norm(c, state)
    return _plain_attend(c, state)


def _run_own(c, s):
    import recommender_sparse_embedding_b200 as R
    if c["kind"] == "embed_lookup":
        return {"out": R.embed_lookup(s["weight"], s["tokens"], scale=c["scale"], padding=PADDING,
                                      out_dtype=DTYPES[c["o"]])}
    if c["kind"] == "embed_grad":
        return {"grad_weight": R.embed_grad(s["tokens"], s["grad"], c["V"], scale=c["scale"], padding=PADDING,
                                            dtype=DTYPES[c["o"]])}
    if c["kind"].startswith("norm"):
        y, mean, rstd = R.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, out_dtype=DTYPES[c["y"]])
        out = {"y": y, "mean": mean, "rstd": rstd}
        if c["kind"] == "norm_train":
            dx, dw, db = R.layer_norm_backward(s["grad"], s["x"], mean, rstd, s["weight"], s["bias"])
            out.update(grad_x=dx, grad_weight=dw, grad_bias=db)
        return out
    a = dict(key_mask=s["mask"])
    o, lse = R.attend(s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"], s["max_q"], s["max_k"], **a)
    out = {"out": o, "lse": lse}
    if c["kind"] == "attend_train":
        dq, dk, dv = R.attend_backward(s["grad"], s["q"], s["k"], s["v"], o, lse, s["q_offsets"], s["k_offsets"],
                                       s["max_q"], s["max_k"], **a)
        out.update(grad_q=dq, grad_k=dk, grad_v=dv)
    return out


def _plain_lookup(c, s):
    t = s["tokens"]
    rows = s["weight"][t.clamp(min=0)].float() * c["scale"]
    return {"out": torch.where((t != PADDING)[:, None], rows, 0.0).to(DTYPES[c["o"]])}


def _plain_grad(c, s):
    t = s["tokens"]
    g = torch.where((t != PADDING)[:, None], s["grad"].float() * c["scale"], 0.0)
    out = torch.zeros((c["V"], c["D"]), dtype=torch.float32, device="cuda")
    return {"grad_weight": out.index_add_(0, t.clamp(min=0), g).to(DTYPES[c["o"]])}


def _plain_norm(c, s):
    x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    xh = xc * rstd
    out = {"y": (xh * w + b).to(DTYPES[c["y"]]), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if c["kind"] == "norm_train":
        dy = s["grad"].float()
        g = dy * w
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        out.update(grad_x=dx.to(s["x"].dtype), grad_weight=(dy * xh).sum(0).to(s["weight"].dtype),
                   grad_bias=dy.sum(0).to(s["bias"].dtype))
    return out


def _bag_rows(offsets, most):
    """Per bag and position: the packed row, and whether the bag is that long."""
    pos = offsets[:-1, None] + torch.arange(most, device=offsets.device)
    return pos, pos < offsets[1:, None]


def _bag_of(offsets, n):
    rows = torch.arange(n, device=offsets.device)
    bag = torch.searchsorted(offsets, rows, right=True) - 1
    return bag, rows - offsets[bag]


def _plain_attend(c, s):
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    G, mq, mk = Hq // Hkv, s["max_q"], s["max_k"]
    nq, nk = s["q"].shape[0], s["k"].shape[0]
    qi, qv = _bag_rows(s["q_offsets"], mq)
    ki, kv = _bag_rows(s["k_offsets"], mk)
    qi, ki = qi.clamp(max=nq - 1), ki.clamp(max=nk - 1)
    if s["mask"] is not None:
        kv = kv & s["mask"][ki]

    def rows_q(x):  # packed queries' rows -> [B, Hkv, G * mq, D]
        x = torch.where(qv[:, :, None, None], x[qi].float(), 0.0)
        return x.view(B, mq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * mq, D)

    def rows_k(x):  # packed keys' rows -> [B, Hkv, mk, D]
        return torch.where(kv[:, :, None, None], x[ki].float(), 0.0).transpose(1, 2)

    bag_q, at_q = _bag_of(s["q_offsets"], nq)

    def packed_q(x, n):  # [B, Hkv, G * mq, n] -> packed queries' rows
        return x.view(B, Hkv, G, mq, n).permute(0, 3, 1, 2, 4)[bag_q, at_q].reshape(nq, Hq, n)

    scale = 1.0 / math.sqrt(D)
    q, k, v = rows_q(s["q"]), rows_k(s["k"]), rows_k(s["v"])
    sc = torch.matmul(q, k.transpose(2, 3)) * scale
    sc = torch.where(kv[:, None, None, :], sc, -math.inf)
    m = sc.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc - m)
    l = p.sum(3, keepdim=True)
    p = p / torch.where(l == 0, 1.0, l)
    o = torch.matmul(p, v)
    out = {"out": packed_q(o, D).to(s["q"].dtype), "lse": packed_q(m + torch.log(l), 1)[:, :, 0]}
    if c["kind"] == "attend_train":
        do = rows_q(s["grad"])
        ds = torch.matmul(do, v.transpose(2, 3))
        ds = p * (ds - (do * o).sum(3, keepdim=True)) * scale
        bag_k, at_k = _bag_of(s["k_offsets"], nk)
        out["grad_q"] = packed_q(torch.matmul(ds, k), D).to(s["q"].dtype)
        out["grad_k"] = torch.matmul(ds.transpose(2, 3), q).transpose(1, 2)[bag_k, at_k].to(s["k"].dtype)
        out["grad_v"] = torch.matmul(p.transpose(2, 3), do).transpose(1, 2)[bag_k, at_k].to(s["v"].dtype)
    return out


# ------------------------------------------------------------------ volumes
def _used_rows(c):
    p = np.arange(1, c["V"] + 1, dtype=np.float64) ** -c["zipf"]
    p /= p.sum()
    return float(-np.expm1(c["N"] * (1 - c["pad"]) * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())


def work(case):
    c = case
    if c["kind"] == "embed_lookup":
        return {"bytes": 8 * c["N"] + _used_rows(c) * c["D"] * BYTES[c["w"]] + c["N"] * c["D"] * BYTES[c["o"]],
                "flops": c["N"] * c["D"]}
    if c["kind"] == "embed_grad":
        return {"bytes": 8 * c["N"] + c["N"] * (1 - c["pad"]) * c["D"] * BYTES[c["g"]]
                + c["V"] * c["D"] * BYTES[c["o"]], "flops": 2 * c["N"] * c["D"]}
    if c["kind"].startswith("norm"):
        n, x, y, w = c["M"] * c["D"], BYTES[c["x"]], BYTES[c["y"]], BYTES[c["w"]]
        nbytes, flops = n * (x + y) + 8 * c["M"] + 2 * c["D"] * w, 8 * n
        if c["kind"] == "norm_train":  # the pass back reads x and the gradient, and writes x's
            nbytes, flops = nbytes + n * (2 * x + y) + 8 * c["M"] + 3 * c["D"] * w, flops + 14 * n
        return {"bytes": nbytes, "flops": flops}
    lq = _lengths(c["B"], c["q_lo"], c["q_hi"]).mean()
    lk = _lengths(c["B"], c["k_lo"], c["k_hi"]).mean()
    nq, nk, t = c["B"] * lq * c["Hq"], c["B"] * lk * c["Hkv"], BYTES[c["t"]]
    macs = c["B"] * lq * lk * (1 - c["masked"]) * c["Hq"] * c["D"]
    nbytes, flops = 2 * (nq + nk) * c["D"] * t + 4 * nq, 4 * macs
    if c["kind"] == "attend_train":  # reads q, k, v, out, its gradient, lse; writes three gradients
        nbytes, flops = nbytes + (4 * nq + 4 * nk) * c["D"] * t + 4 * nq, flops + 10 * macs
    return {"bytes": float(nbytes), "flops": float(flops)}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "embed_lookup":
        out = torch.zeros((c["N"], c["D"]), dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["tokens"] >= 0)[:, 0]
        out[at] = s["weight"].double()[s["tokens"][at]] * c["scale"]
        return {"out": out}
    if c["kind"] == "embed_grad":
        # sorted by token, the running sums' differences at the tokens' ends
        at = torch.nonzero(s["tokens"] >= 0)[:, 0]
        t, order = torch.sort(s["tokens"][at])
        ends = torch.searchsorted(t, torch.arange(c["V"] + 1, device="cuda"))
        out = torch.empty((c["V"], c["D"]), dtype=torch.float64, device="cuda")
        for d in range(0, c["D"], 32):
            run_sum = torch.cat([torch.zeros((1, min(32, c["D"] - d)), dtype=torch.float64, device="cuda"),
                                 s["grad"][:, d:d + 32].double()[at[order]].cumsum(0)])
            out[:, d:d + 32] = (run_sum[ends[1:]] - run_sum[ends[:-1]]) * c["scale"]
        return {"grad_weight": out}
    if c["kind"].startswith("norm"):
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS).rsqrt()
        w = s["weight"].double()
        x = x.sub_(mean[:, None]).mul_(rstd[:, None])
        out = {"y": x * w + s["bias"].double(), "mean": mean, "rstd": rstd}
        if c["kind"] == "norm_train":
            dy = s["grad"].double()
            out["grad_weight"], out["grad_bias"] = torch.einsum("md,md->d", dy, x), torch.einsum("md->d", dy)
            dy = dy.mul_(w)
            a, b = torch.einsum("md->m", dy) / c["D"], torch.einsum("md,md->m", dy, x) / c["D"]
            out["grad_x"] = dy.sub_(a[:, None]).sub_(x.mul_(b[:, None])).mul_(rstd[:, None])
        return out
    qo, ko = s["q_offsets"].tolist(), s["k_offsets"].tolist()
    G, inv = c["Hq"] // c["Hkv"], c["D"] ** -0.5
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    out = {"out": torch.zeros_like(q), "lse": torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")}
    if c["kind"] == "attend_train":
        do = s["grad"].double()
        out.update(grad_q=torch.zeros_like(q), grad_k=torch.zeros_like(k), grad_v=torch.zeros_like(v))
    for b in range(c["B"]):
        rows, keys = slice(qo[b], qo[b + 1]), torch.arange(ko[b], ko[b + 1], device="cuda")
        if s["mask"] is not None:
            keys = keys[s["mask"][keys]]
        if qo[b] == qo[b + 1] or keys.numel() == 0:
            continue
        kb, vb = k[keys].permute(1, 0, 2), v[keys].permute(1, 0, 2)  # [Hkv, n, D]
        qb = q[rows].unflatten(1, (c["Hkv"], G)).permute(1, 2, 0, 3).flatten(1, 2)  # [Hkv, G * m, D]

        def back(x):  # [Hkv, G * m, ...] -> [m, Hq, ...]
            return x.unflatten(1, (G, -1)).flatten(0, 1).transpose(0, 1)

        sc = qb @ kb.mT * inv
        lse = torch.logsumexp(sc, 2)
        p = torch.exp(sc - lse[:, :, None])
        ob = p @ vb
        out["out"][rows], out["lse"][rows] = back(ob), back(lse)
        if c["kind"] == "attend_train":
            gb = do[rows].unflatten(1, (c["Hkv"], G)).permute(1, 2, 0, 3).flatten(1, 2)
            ds = p * (gb @ vb.mT - (gb * ob).sum(2, keepdim=True)) * inv
            out["grad_q"][rows] = back(ds @ kb)
            out["grad_k"][keys] = (ds.mT @ qb).permute(1, 0, 2)
            out["grad_v"][keys] = (p.mT @ gb).permute(1, 0, 2)
    return out
