"""Cases of the token embedding (lookup with scaling, gradient by sorted tokens)
and of the jagged attention (forward, backward), each in a plain form and as a
call of the framework.

A case names its operator in "op":

lookup     out[i] = scale * table[ids[i]], another output type allowed
grad       g[v] = scale * the sum of dout[i] over the tokens i with ids[i] == v;
           the padding id takes no part
attention  softmax attention inside every sample of a jagged batch: a sample's
           last tokens are candidates, which see the history and themselves;
           history tokens see the history, up to themselves where `causal`
backward   its gradients of q, k and v
"""

import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _bytes(name):
    return 4 if name == "f32" else 2


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one token at serving time: latency only
        dict(name="lookup, one token", op="lookup", n=1, rows=100_000, dim=2048, zipf=1.05,
             table="bf16", out="bf16"),
        # a training batch's tokens, rows of a vocabulary
        dict(name="lookup, a batch", op="lookup", n=32_768, rows=100_000, dim=1024, zipf=1.05,
             table="bf16", out="bf16"),
        # fp32 master rows looked up into bf16 activations, odd sizes
        dict(name="lookup, large", op="lookup", n=200_003, rows=1_000_000, dim=636, zipf=1.1,
             table="f32", out="bf16"),
        # the smallest batch: 64 samples' last tokens and a few more
        dict(name="grad, few tokens", op="grad", n=300, rows=100_000, dim=64, zipf=1.05, pad=0,
             dout="f32", grad="f32"),
        # an ordinary training batch
        dict(name="grad, a batch", op="grad", n=16_384, rows=32_000, dim=1024, zipf=1.05, pad=0,
             dout="bf16", grad="f32"),
        # a large batch with hot rows of tens of thousands of tokens
        dict(name="grad, large", op="grad", n=262_139, rows=131_072, dim=1000, zipf=1.2, pad=7,
             dout="bf16", grad="bf16"),
        # many short histories with a few candidates
        dict(name="attention, short", op="attention", n=64, longest=256, law="lognormal", cand=4,
             heads=2, kv_heads=2, dim=32, type="bf16", causal=True, masked=0.0, fused=False),
        # skewed histories, shared key heads, dropped ids, one fused projection
        dict(name="attention, ordinary", op="attention", n=128, longest=1024, law="pareto", cand=8,
             heads=8, kv_heads=2, dim=64, type="bf16", causal=True, masked=0.02, fused=True),
        # a few long histories
        dict(name="attention, long", op="attention", n=4, longest=8192, law="equal", cand=0,
             heads=4, kv_heads=4, dim=128, type="bf16", causal=True, masked=0.0, fused=False),
        # the same three in training's other direction, with other heads and types
        dict(name="backward, short", op="backward", n=64, longest=250, law="lognormal", cand=4,
             heads=2, kv_heads=1, dim=40, type="f16", causal=False, masked=0.05, fused=False),
        dict(name="backward, ordinary", op="backward", n=128, longest=1024, law="pareto", cand=8,
             heads=8, kv_heads=2, dim=64, type="bf16", causal=True, masked=0.02, fused=True),
        dict(name="backward, long", op="backward", n=2, longest=8192, law="equal", cand=0,
             heads=8, kv_heads=2, dim=128, type="bf16", causal=True, masked=0.0, fused=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["lookup", "grad", "attention", "backward"])
    if op in ("lookup", "grad"):
        dim = _log(rng, 16, 4096)
        if rng.random() < 0.7:  # most rows hold whole 16-byte pieces
            dim = max(16, dim // 8 * 8)
        if op == "lookup":
            return dict(op=op, n=_log(rng, 1, min(262_144, (1 << 27) // dim)),
                        rows=_log(rng, 1000, min(1_000_000, (1 << 29) // dim)), dim=dim,
                        zipf=rng.choice([1.05, 1.1, 1.2]), table=rng.choice(["f32", "bf16", "f16"]),
                        out=rng.choice(["f32", "bf16", "f16"]))
        return dict(op=op, n=_log(rng, 1, min(262_144, (1 << 27) // dim)),
                    rows=_log(rng, 500, min(262_144, (1 << 27) // dim)), dim=dim,
                    zipf=rng.choice([1.05, 1.1, 1.2]), pad=rng.choice([-1, 0, 7]),
                    dout=rng.choice(["f32", "bf16", "f16"]), grad=rng.choice(["f32", "bf16", "f16"]))
    heads, group = rng.choice([1, 2, 4, 6, 8, 16]), rng.choice([1, 1, 2, 4])
    if heads % group:
        group = 1
    longest = _log(rng, 1, 8192)
    n = _log(rng, 1, max(1, min(512, (1 << 28) // (heads * longest * longest))))
    return dict(op=op, n=n, longest=longest, law=rng.choice(["lognormal", "pareto", "equal"]),
                cand=rng.choice([0, 4, 16]), heads=heads, kv_heads=heads // group,
                dim=rng.choice([16, 32, 40, 64, 64, 96, 128, 128]), type=rng.choice(["bf16", "f16"]),
                causal=rng.random() < 0.7, masked=rng.choice([0.0, 0.0, 0.02, 0.2]),
                fused=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _zipf_ids(n, rows, s, g):
    """Bounded power law over ranks 1..rows, ranks spread over the rows."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = (((rows + 1.0) ** (1 - s) - 1) * u + 1) ** (1 / (1 - s))
    rank = (rank.floor().to(torch.int64) - 1).clamp_(0, rows - 1)
    step = 2654435761 % rows | 1
    while math.gcd(step, rows) != 1:
        step += 2
    return (rank * step + 12345) % rows


def _distinct(n, rows, s):
    """How many rows n draws of that law meet on average."""
    r = np.arange(1, rows + 1, dtype=np.float64)
    cdf = ((np.append(r, rows + 1.0)) ** (1 - s) - 1) / ((rows + 1.0) ** (1 - s) - 1)
    p = np.diff(cdf)
    return float(-np.expm1(n * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())


def _shape(case):
    """Lengths and candidate counts of the samples, shortest first."""
    n, longest = case["n"], case["longest"]
    at = (np.arange(n) + 0.5) / n
    if case["law"] == "equal":
        x = np.full(n, float(longest))
    elif case["law"] == "lognormal":  # median a quarter of the longest
        z = torch.erfinv(torch.from_numpy(2 * at - 1)).numpy() * math.sqrt(2)
        x = longest / 4 * np.exp(z)
    else:
        x = longest / 6 * (1 - at) ** (-1 / 1.2)
    lens = np.clip(np.ceil(x), 1, longest).astype(np.int64)
    cand = np.zeros(n, np.int64)
    if case["cand"]:
        cand = np.minimum(1 + np.arange(n) % case["cand"], lens)
    return lens, cand


def _prepare_tokens(case, g):
    ids = _zipf_ids(case["n"], case["rows"], case["zipf"], g)
    if case["op"] == "lookup":
        w = torch.empty(case["rows"], case["dim"], device="cuda", dtype=_TYPES[case["table"]])
        w.normal_(0, 0.02, generator=g)
        return dict(case=case, ids=ids, weight=w, scale=math.sqrt(case["dim"]),
                    dtype=_TYPES[case["out"]])
    dout = torch.empty(case["n"], case["dim"], device="cuda", dtype=_TYPES[case["dout"]])
    dout.normal_(0, 0.01, generator=g)
    return dict(case=case, ids=ids, dout=dout, rows=case["rows"], pad=case["pad"],
                scale=math.sqrt(case["dim"]), dtype=_TYPES[case["grad"]])


def _prepare_attention(case, seed, g):
    lens, cand = _shape(case)
    order = np.random.default_rng(int(seed)).permutation(case["n"])
    lens, cand = lens[order], cand[order]
    offsets = np.concatenate([[0], np.cumsum(lens)])
    n_tok, hq, hk, d = int(offsets[-1]), case["heads"], case["kv_heads"], case["dim"]
    t = _TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(t)

    if case["fused"]:  # q, k and v are views of one projection's output
        qkv = normal(n_tok, hq + 2 * hk, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    else:
        q, k, v = normal(n_tok, hq, d), normal(n_tok, hk, d), normal(n_tok, hk, d)
    s = dict(case=case, q=q, k=k, v=v, scale=1 / math.sqrt(d), causal=case["causal"],
             offsets=torch.from_numpy(offsets).cuda(), n_cand=None, valid=None,
             longest=int(lens.max()))
    if case["cand"]:
        s["n_cand"] = torch.from_numpy(cand.astype(np.int32)).cuda()
    if case["masked"]:
        s["valid"] = (torch.rand(n_tok, generator=g, device="cuda") >= case["masked"]).to(torch.uint8)
    if case["op"] == "backward":
        s["dout"] = normal(n_tok, hq, d)
        s["out"], s["lse"] = _attention(s)  # what the forward pass left behind
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] in ("lookup", "grad"):
        return _prepare_tokens(case, g)
    return _prepare_attention(case, seed, g)


# ---------------------------------------------------------------- one pass


def run(state):
    op = state["case"]["op"]
    if own:
        from jagged_embedding_sparse_amd import lib
        if op == "lookup":
            return lib.fs_token_lookup(state["weight"], state["ids"], scale=state["scale"],
                                       dtype=state["dtype"])
        if op == "grad":
            uq = lib.fs_token_sort(state["ids"], state["rows"], padding_id=state["pad"])
            return lib.fs_token_grad(uq, state["dout"], state["rows"], scale=state["scale"],
                                     dtype=state["dtype"])
        args = dict(n_cand=state["n_cand"], valid=state["valid"], causal=state["causal"],
                    scale=state["scale"])
        if op == "attention":
            out, lse = lib.fs_jagged_attention(state["q"], state["k"], state["v"],
                                               state["offsets"], **args)
            return {"out": out, "lse": lse}
        dq, dk, dv = lib.fs_jagged_attention_backward(state["q"], state["k"], state["v"],
                                                      state["out"], state["lse"], state["dout"],
                                                      state["offsets"], **args)
        return {"dq": dq, "dk": dk, "dv": dv}
    if op == "lookup":
        return (state["weight"][state["ids"]].float() * state["scale"]).to(state["dtype"])
    if op == "grad":
        keep = (state["ids"] != state["pad"]).float() * state["scale"]
        g = torch.zeros(state["rows"], state["dout"].shape[1], device="cuda")
        return g.index_add_(0, state["ids"], state["dout"].float() * keep[:, None]).to(state["dtype"])
    if op == "attention":
        out, lse = _attention(state)
        return {"out": out, "lse": lse}
    return _backward(state)


def _padded(state):
    """Where the tokens of a padded batch lie, and which of them see which."""
    off, n = state["offsets"], state["case"]["n"]
    i = torch.arange(state["longest"], device="cuda")
    lens = off[1:] - off[:-1]
    real = i < lens[:, None]
    at = torch.where(real, off[:-1, None] + i, 0)
    live = real if state["valid"] is None else real & (state["valid"][at] != 0)
    hist = lens if state["n_cand"] is None else lens - state["n_cand"]
    sees = (i < hist[:, None])[:, None, :].expand(n, len(i), len(i))
    if state["causal"]:
        sees = sees & (i[None, :] <= i[:, None])
    sees = (sees | (i[None, :] == i[:, None])) & live[:, :, None] & live[:, None, :]
    return at, real, sees[:, None]


def _heads_first(x, at, group=1):
    return x[at].float().transpose(1, 2).repeat_interleave(group, 1).contiguous()


def _scores(state, at, sees, q, k):
    s = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(state["scale"])
    s.masked_fill_(~sees, -math.inf)
    top = s.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    lse = (top + total.log())[..., 0]
    return p.div_(torch.where(total == 0, 1.0, total)), lse


def _attention(state):
    at, real, sees = _padded(state)
    group = state["q"].shape[1] // state["k"].shape[1]
    q = _heads_first(state["q"], at)
    k, v = _heads_first(state["k"], at, group), _heads_first(state["v"], at, group)
    p, lse = _scores(state, at, sees, q, k)
    out = torch.matmul(p, v).transpose(1, 2)[real].to(state["q"].dtype)
    return out, lse.transpose(1, 2)[real].t().contiguous()


def _backward(state):
    at, real, sees = _padded(state)
    hk, d, dtype = state["k"].shape[1], state["q"].shape[2], state["q"].dtype
    group = state["q"].shape[1] // hk
    q, do = _heads_first(state["q"], at), _heads_first(state["dout"], at)
    do = do * real[:, None, :, None]
    k, v = _heads_first(state["k"], at, group), _heads_first(state["v"], at, group)
    p, _ = _scores(state, at, sees, q, k)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
    ds = torch.matmul(do, v.transpose(2, 3).contiguous())
    ds = ds.sub_((ds * p).sum(3, keepdim=True)).mul_(p).mul_(state["scale"])
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q)

    def back(x, heads):
        x = x.unflatten(1, (heads, -1)).sum(2) if heads != x.shape[1] else x
        return x.transpose(1, 2)[real].to(dtype)

    return {"dq": back(dq, hk * group), "dk": back(dk, hk), "dv": back(dv, hk)}


# ---------------------------------------------------------------- least work


def _pairs(case):
    lens, cand = (x.astype(np.float64) for x in _shape(case))
    h = lens - cand
    pairs = (h * (h + 1) / 2 if case["causal"] else h * h) + cand * (h + 1)
    return float(pairs.sum()) * (1 - case["masked"]) ** 2


def work(case):
    if case["op"] in ("lookup", "grad"):
        n, rows, d = case["n"], case["rows"], case["dim"]
        if case["op"] == "lookup":
            return {"bytes": 8 * n + n * d * _bytes(case["out"])
                    + _distinct(n, rows, case["zipf"]) * d * _bytes(case["table"]), "flops": n * d}
        return {"bytes": 8 * n + n * d * _bytes(case["dout"]) + rows * d * _bytes(case["grad"]),
                "flops": 2 * n * d}
    tokens = float(_shape(case)[0].sum())
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    times = 2 if case["op"] == "attention" else 4  # q, out / q, out, dout, dq; the same for k, v
    return {"bytes": tokens * (times * (hq + hk) * d * 2 + 4 * hq),
            "flops": (2 * times + (2 if times == 4 else 0)) * d * hq * _pairs(case)}


# ---------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lookup":
        return s["weight"].index_select(0, s["ids"]).double() * s["scale"]
    if case["op"] == "grad":
        ids, order = s["ids"].sort(stable=True)
        d = s["dout"].double()[order] * s["scale"]
        d[ids == s["pad"]] = 0
        g = torch.zeros(s["rows"], d.shape[1], device="cuda", dtype=torch.float64)
        return g.index_put_((ids,), d, accumulate=True)
    group = case["heads"] // case["kv_heads"]
    off = s["offsets"].tolist()
    got = []
    for b in range(case["n"]):
        lo, hi = off[b], off[b + 1]
        c = int(s["n_cand"][b]) if s["n_cand"] is not None else 0
        got.append(_exact_sample(s, lo, hi, hi - lo - c, group))
    names = ("out", "lse") if case["op"] == "attention" else ("dq", "dk", "dv")
    return {name: torch.cat([x[i] for x in got], 1 if name == "lse" else 0)
            for i, name in enumerate(names)}


def _exact_sample(s, lo, hi, hist, group):
    q, k, v = (s[x][lo:hi].double().permute(1, 0, 2) for x in "qkv")
    k, v = (x[:, None].expand(-1, group, -1, -1).reshape(-1, hi - lo, x.shape[2]) for x in (k, v))
    i = torch.arange(hi - lo, device="cuda")
    row, col = i[:, None], i[None, :]
    sees = (col < hist) & ((col <= row) | (not s["causal"])) | (col == row)
    if s["valid"] is not None:
        ok = s["valid"][lo:hi].bool()
        sees = sees & ok[:, None] & ok[None, :]
    a = (q @ k.mT.contiguous() * s["scale"]).masked_fill(~sees, -math.inf)
    lse = torch.logsumexp(a, 2)
    p = torch.exp(a - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    if "dout" not in s:
        return (p @ v).permute(1, 0, 2), lse
    do = s["dout"][lo:hi].double().permute(1, 0, 2)
    dp = do @ v.mT.contiguous()
    ds = p * (dp - (p * dp).sum(2, keepdim=True)) * s["scale"]
    dq, dk, dv = ds @ k, ds.mT.contiguous() @ q, p.mT.contiguous() @ do
    dk, dv = (x.reshape(-1, group, *x.shape[1:]).sum(1) for x in (dk, dv))
    return dq.permute(1, 0, 2), dk.permute(1, 0, 2), dv.permute(1, 0, 2)
