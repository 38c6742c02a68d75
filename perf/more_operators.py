"""Cases of the layer norm and of the two losses over a vocabulary's table, each
with its gradients, in a plain form and as calls of the framework.

A case names its operator in "op":

norm           out = (x - mean) rstd weight + bias, row by row; mean and rstd come out too
norm back      gradients of x, weight and bias
loss           softmax cross entropy of every token against the table: with z = scale x w^T,
               lse_i = log(sum_v exp z_iv) and loss_i = lse_i - z_i,label;
               tokens with the padding id as their label take no part
loss back      gradients of x and w for given gradients of the tokens' losses
distill        the same softmax against a teacher's top logits: q_i is the softmax of
               scale * teacher over a token's entries, loss_i = sum_k q_ik
               (log q_ik - z_i,id(k) + lse_i); entries with the padding id take no part
distill back   gradients of x and w
"""

import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_PAD = -1
_EPS = 1e-5


def _bytes(name):
    return 4 if name == "f32" else 2


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one token at serving time: latency only
        dict(name="norm: one token", op="norm", n=1, dim=2048, x="bf16", out="bf16", param="bf16"),
        # a training batch's fp32 residual stream, normed into bf16 activations
        dict(name="norm: a batch", op="norm", n=32_768, dim=1024, x="f32", out="bf16", param="f32"),
        # a few samples' tokens, narrow rows
        dict(name="norm back: few tokens", op="norm back", n=300, dim=64, x="f32", out="f32",
             param="f32"),
        # a large batch, odd sizes, everything in 16 bits
        dict(name="norm back: large", op="norm back", n=65_537, dim=1000, x="bf16", out="bf16",
             param="bf16"),
        # the samples' last tokens scored against a vocabulary: one pass over its rows
        dict(name="loss: few tokens", op="loss", n=17, rows=100_000, dim=256, type="bf16", zipf=1.05,
             masked=0.0, scale=1.0),
        # a training batch, a tenth of its tokens without a label
        dict(name="loss: a batch", op="loss", n=16_384, rows=100_000, dim=1024, type="bf16",
             zipf=1.05, masked=0.1, scale=1.0),
        # a small batch, fp16
        dict(name="loss back: few tokens", op="loss back", n=64, rows=32_000, dim=64, type="f16",
             zipf=1.05, masked=0.2, scale=1.0),
        # the largest: a training batch against a large vocabulary
        dict(name="loss back: large", op="loss back", n=16_384, rows=131_072, dim=1024, type="bf16",
             zipf=1.05, masked=0.0, scale=1.0),
        # a short batch with a few entries for each token, temperature 2
        dict(name="distill: short", op="distill", n=128, rows=50_000, dim=256, type="f16", zipf=1.1,
             masked=0.0, top=16, teacher="f16", scale=0.5),
        # an ordinary batch
        dict(name="distill: a batch", op="distill", n=8192, rows=32_000, dim=1024, type="bf16",
             zipf=1.05, masked=0.05, top=64, teacher="bf16", scale=1.0),
        # odd sizes, some entries missing
        dict(name="distill back: short", op="distill back", n=499, rows=10_007, dim=200, type="f16",
             zipf=1.1, masked=0.1, top=8, teacher="f32", scale=0.5),
        dict(name="distill back: a batch", op="distill back", n=8192, rows=65_536, dim=768,
             type="bf16", zipf=1.05, masked=0.05, top=32, teacher="f32", scale=1.0),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm back", "loss", "loss back", "distill", "distill back"])
    if op.startswith("norm"):
        dim = _log(rng, 16, 8192)
        if rng.random() < 0.7:  # most rows hold whole 16-byte pieces
            dim = dim // 8 * 8
        x = rng.choice(["f32", "bf16", "f16"])
        return dict(op=op, n=_log(rng, 1, min(131_072, (1 << 26) // dim)), dim=dim, x=x,
                    out=rng.choice([x, x, "f32", "bf16"]), param=rng.choice([x, "f32"]))
    dim = _log(rng, 32, 2048)
    if rng.random() < 0.8:  # most widths are of whole 16-byte pieces, and round
        dim = max(32, dim // 64 * 64) if rng.random() < 0.6 else dim // 8 * 8
    rows = _log(rng, 300, 200_000)
    n = _log(rng, 1, min(16_384, (1 << 31) // rows, (1 << 41) // (rows * dim)))
    case = dict(op=op, n=n, rows=rows, dim=dim, type=rng.choice(["bf16", "bf16", "f16"]),
                zipf=rng.choice([1.05, 1.1, 1.2]), masked=rng.choice([0.0, 0.0, 0.1, 0.6]),
                scale=rng.choice([1.0, 1.0, 0.5, 1.5]))
    if op.startswith("distill"):
        case.update(top=_log(rng, 1, 128), teacher=rng.choice(["f32", "bf16", "f16"]))
    return case


# ---------------------------------------------------------------- inputs


def _zipf_ranks(n, rows, s, g):
    """Bounded power law over ranks 0 .. rows - 1."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = (((rows + 1.0) ** (1 - s) - 1) * u + 1) ** (1 / (1 - s))
    return (rank.floor().to(torch.int64) - 1).clamp_(0, rows - 1)


def _spread(rank, rows):
    """Ranks to rows, one to one."""
    step = 2654435761 % rows | 1
    while math.gcd(step, rows) != 1:
        step += 2
    return (rank * step + 12345) % rows


def _prepare_norm(case, g):
    n, dim = case["n"], case["dim"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # a residual stream: columns of their own offset, a few of them large
    at = 0.5 * normal(dim)
    at[:: 97] *= 20
    s = dict(case=case, x=(normal(n, dim).mul_(2).add_(at)).to(_TYPES[case["x"]]),
             weight=(1 + 0.2 * normal(dim)).to(_TYPES[case["param"]]),
             bias=(0.1 * normal(dim)).to(_TYPES[case["param"]]), dtype=_TYPES[case["out"]])
    if case["op"] == "norm back":
        s["mean"], s["rstd"] = _norm(s)[1:]  # what the forward pass left behind
        s["dout"] = normal(n, dim).mul_(0.01).to(s["dtype"])
    return s


def _prepare_loss(case, g):
    n, rows, dim, t = case["n"], case["rows"], case["dim"], _TYPES[case["type"]]
    top = case.get("top", 1)
    w = torch.empty(rows, dim, device="cuda").normal_(0, 2 / math.sqrt(dim), generator=g).to(t)
    # a token's entries: neighbours in rank, the first of them drawn by the power law
    rank = _zipf_ranks(n, rows, case["zipf"], g)[:, None] + torch.arange(min(top, rows), device="cuda")
    ids = _spread(rank % rows, rows)
    # some tokens are close to their label's row, others are not
    near = 3 * torch.rand(n, 1, generator=g, device="cuda")
    x = torch.randn(n, dim, generator=g, device="cuda").add_(near * w[ids[:, 0]].float()).to(t)
    off = torch.rand(n, generator=g, device="cuda") < case["masked"]
    s = dict(case=case, x=x, weight=w, scale=case["scale"])
    if case["op"].startswith("loss"):
        s["labels"] = torch.where(off, _PAD, ids[:, 0])
    else:
        k = torch.arange(ids.shape[1], device="cuda")
        s["teacher"] = (12 - 3 * torch.log1p(k) + 0.5 * torch.randn(ids.shape, generator=g, device="cuda")
                        ).to(_TYPES[case["teacher"]])
        # a quarter of the tokens has fewer entries
        few = torch.rand(n, generator=g, device="cuda") < 0.25
        count = torch.randint(1, ids.shape[1] + 1, (n,), generator=g, device="cuda")
        count = torch.where(off, 0, torch.where(few, count, ids.shape[1]))
        s["ids"] = torch.where(k < count[:, None], ids, _PAD)
    if case["op"].endswith("back"):
        s["dloss"] = (0.5 + torch.rand(n, generator=g, device="cuda")) / n
        if case["op"] == "loss back":
            s["lse"] = _loss(s)["lse"]
        else:
            left = _distill(s)
            s["lse"], s["logits"] = left["lse"], left["logits"]
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return (_prepare_norm if case["op"].startswith("norm") else _prepare_loss)(case, g)


# ---------------------------------------------------------------- one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    if op == "norm":
        out, mean, rstd = _norm(state)
        return {"out": out, "mean": mean, "rstd": rstd}
    if op == "norm back":
        return _norm_back(state)
    if op == "loss":
        return _loss(state)
    if op == "loss back":
        return _loss_back(state)
    if op == "distill":
        return _distill(state)
    return _distill_back(state)


def _own(op, s):
    from jagged_embedding_sparse_amd import lib
    if op == "norm":
        out, mean, rstd = lib.fs_layer_norm(s["x"], s["weight"], s["bias"], eps=_EPS, dtype=s["dtype"])
        return {"out": out, "mean": mean, "rstd": rstd}
    if op == "norm back":
        dx, dweight, dbias = lib.fs_layer_norm_backward(s["x"], s["mean"], s["rstd"], s["dout"],
                                                        s["weight"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    kw = dict(scale=s["scale"], padding_id=_PAD)
    if op == "loss":
        loss, lse = lib.fs_token_loss(s["x"], s["weight"], s["labels"], **kw)
        return {"loss": loss, "lse": lse}
    if op == "loss back":
        dx, dweight = lib.fs_token_loss_backward(s["x"], s["weight"], s["labels"], s["lse"],
                                                 s["dloss"], **kw)
        return {"dx": dx, "dweight": dweight}
    if op == "distill":
        loss, lse, logits = lib.fs_token_distill(s["x"], s["weight"], s["ids"], s["teacher"], **kw)
        return {"loss": loss, "lse": lse, "logits": logits}
    dx, dweight = lib.fs_token_distill_backward(s["x"], s["weight"], s["ids"], s["teacher"], s["lse"],
                                                s["logits"], s["dloss"], **kw)
    return {"dx": dx, "dweight": dweight}


def _norm(s):
    x = s["x"].float()
    mean = x.sum(1) / x.shape[1]
    x = x - mean[:, None]
    rstd = torch.rsqrt((x * x).sum(1) / x.shape[1] + _EPS)
    out = x.mul_(rstd[:, None]).mul_(s["weight"].float()).add_(s["bias"].float())
    return out.to(s["dtype"]), mean, rstd


def _norm_back(s):
    x, dout, dim = s["x"].float(), s["dout"].float(), s["x"].shape[1]
    hat = (x - s["mean"][:, None]).mul_(s["rstd"][:, None])
    g = dout * s["weight"].float()
    dx = g - (g.sum(1, keepdim=True) / dim) - hat * ((g * hat).sum(1, keepdim=True) / dim)
    dx = dx.mul_(s["rstd"][:, None]).to(s["x"].dtype)
    t = s["weight"].dtype
    return {"dx": dx, "dweight": (dout * hat).sum(0).to(t), "dbias": dout.sum(0).to(t)}


def _scores(s):
    """Logits of all rows, and what their softmax divides by."""
    z = torch.mm(s["x"].float(), s["weight"].float().t()).mul_(s["scale"])
    top = z.amax(1)
    return z, top + torch.exp(z - top[:, None]).sum(1).log_()


def _loss(s):
    z, lse = _scores(s)
    live = s["labels"] != _PAD
    at = torch.where(live, s["labels"], 0)
    loss = lse - z.gather(1, at[:, None])[:, 0]
    return {"loss": torch.where(live, loss, 0.0), "lse": torch.where(live, lse, 0.0)}


def _teacher(s):
    """The teacher's softmax over a token's entries, its logarithm (0 for no entry)
    and which tokens take part."""
    on = s["ids"] != _PAD
    t = (s["teacher"].float() * s["scale"]).masked_fill_(~on, -math.inf)
    top = t.amax(1, keepdim=True)
    t = t - torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(t)
    total = e.sum(1, keepdim=True)
    live = total[:, 0] > 0
    total = torch.where(total > 0, total, 1.0)
    return on, e / total, (t - total.log()).masked_fill_(~on, 0.0), live


def _distill(s):
    z, lse = _scores(s)
    on, q, logq, live = _teacher(s)
    at = z.gather(1, torch.where(on, s["ids"], 0)).masked_fill_(~on, 0.0)
    loss = (q * (logq - at + lse[:, None])).sum(1)
    return {"loss": torch.where(live, loss, 0.0), "lse": torch.where(live, lse, 0.0), "logits": at}


def _gradients(s, d, live):
    d.mul_((s["dloss"] * s["scale"])[:, None]).masked_fill_(~live[:, None], 0.0)
    dx = torch.mm(d, s["weight"].float()).to(s["x"].dtype)
    dw = torch.mm(d.t(), s["x"].float()).to(s["weight"].dtype)
    return {"dx": dx, "dweight": dw}


def _softmax(s):
    z = torch.mm(s["x"].float(), s["weight"].float().t()).mul_(s["scale"])
    return z.sub_(s["lse"][:, None]).exp_()


def _loss_back(s):
    live = s["labels"] != _PAD
    at = torch.where(live, s["labels"], 0)[:, None]
    d = _softmax(s)
    d.scatter_(1, at, d.gather(1, at) - 1)
    return _gradients(s, d, live)


def _distill_back(s):
    on, q, _, live = _teacher(s)
    d = _softmax(s)
    d.scatter_add_(1, torch.where(on, s["ids"], 0), -q)  # no entry adds nothing
    return _gradients(s, d, live)


# ---------------------------------------------------------------- least work


def work(case):
    n, dim = case["n"], case["dim"]
    if case["op"].startswith("norm"):
        x, out, param = _bytes(case["x"]), _bytes(case["out"]), _bytes(case["param"])
        if case["op"] == "norm":
            return {"bytes": n * dim * (x + out) + 2 * dim * param + 8 * n, "flops": 7 * n * dim}
        return {"bytes": n * dim * (2 * x + out) + 3 * dim * param + 8 * n, "flops": 13 * n * dim}
    rows, top, live = case["rows"], case.get("top", 1), n * (1 - case["masked"])
    entry = 8 + (_bytes(case["teacher"]) + 4 if "top" in case else 0)
    read = (live + rows) * dim * 2 + n * top * entry
    if case["op"].endswith("back"):
        return {"bytes": read + (n + rows) * dim * 2 + 8 * n, "flops": 6 * live * rows * dim}
    return {"bytes": read + 8 * n, "flops": 2 * live * rows * dim}


# ---------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    parts, dw, step = [], 0, max(1, (1 << 28) // case["rows"])
    w = s["weight"].double()
    for lo in range(0, case["n"], step):
        got, more = _exact_rows(s, slice(lo, lo + step), w)
        parts.append(got)
        dw = dw + more if more is not None else dw
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["op"].endswith("back"):
        out["dweight"] = dw
    return out


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    if "dout" not in s:
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + _EPS) ** -0.5
        return {"out": (x - mean[:, None]) * rstd[:, None] * w + s["bias"].double(), "mean": mean,
                "rstd": rstd}
    rstd, dout = s["rstd"].double()[:, None], s["dout"].double()
    hat = (x - s["mean"].double()[:, None]) * rstd
    g = dout * w
    dx = rstd * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    return {"dx": dx, "dweight": (hat * dout).sum(0), "dbias": dout.sum(0)}


def _exact_rows(s, at, w):
    """A slice of the tokens: their outputs, and what they add to the table's gradient."""
    x = s["x"][at].double()
    z = x @ w.mT * s["scale"]
    if "labels" in s:
        ids = s["labels"][at, None]
        on = ids >= 0
        q = on.double()
    else:
        ids = s["ids"][at]
        on = ids >= 0
        t = (s["teacher"][at].double() * s["scale"]).masked_fill(~on, -math.inf)
        q = torch.softmax(t, 1).masked_fill(~on.any(1, keepdim=True), 0.0)
    live = on.any(1)
    idx = torch.where(on, ids, 0)
    if "dloss" in s:
        d = torch.exp(z - s["lse"][at].double()[:, None])
        d.scatter_add_(1, idx, -q)
        d *= (live * s["dloss"][at].double() * s["scale"])[:, None]
        return {"dx": d @ w}, d.mT @ x
    lse = torch.logsumexp(z, 1)
    zk = z.gather(1, idx)
    own_part = torch.where(q > 0, q * q.clamp_min(1e-300).log(), 0.0).sum(1)
    loss = own_part - (q * zk).sum(1) + lse
    got = {"loss": torch.where(live, loss, 0.0), "lse": torch.where(live, lse, 0.0)}
    if "labels" not in s:
        got["logits"] = torch.where(on, zk, 0.0)
    return got, None
