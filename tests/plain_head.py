"""Plain 64-bit forms of the layer norm and of the losses over a vocabulary's
table, on the CPU, and how far a result rounded to fewer bits may be from them
(plain_ops has how bounds count roundings)."""

import math

import torch

from plain_ops import U32, tiny, u

# A row's sum in the kernels: a lane's values, 6 exchanges inside a wave, a row's waves, and
# the division by dim. Values and waves are 32 together at most: 16 and 16 (1024 lanes of two
# pieces of 8 or four of 4), 24 and 8 (512 lanes of three pieces of 8).
NORM_STEPS = 16 + 6 + 16 + 2


def norm(x, weight, bias, eps, dtype):
    """dict of (value, bound) of out (in dtype), mean and rstd."""
    x, dim = x.double(), x.shape[1]
    w = torch.ones(dim, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(dim, dtype=torch.float64) if bias is None else bias.double()
    mean = x.mean(1, keepdim=True)
    v = x - mean
    var = (v * v).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    out = v * rstd * w + b
    e_mean = NORM_STEPS * U32 * x.abs().mean(1, keepdim=True)
    e_v = e_mean + U32 * v.abs()
    e_var = (2 * v.abs() * e_v + e_v * e_v).mean(1, keepdim=True) + (NORM_STEPS + 1) * U32 * var
    # of rstd: half the sum's relative error, the sum with eps, root and quotient
    r = 0.5 * e_var / (var + eps) * 1.01 + 4 * U32
    bound = ((e_v + v.abs() * r) * rstd * w.abs() + 3 * U32 * (v * rstd * w).abs() + U32 * out.abs())
    return dict(out=(out, bound * (1 + u(dtype)) + u(dtype) * out.abs() + tiny(dtype)),
                mean=(mean[:, 0], e_mean[:, 0] + 1e-40), rstd=(rstd[:, 0], (r * rstd)[:, 0]))


def norm_backward(x, mean, rstd, dout, weight, dtype, param):
    """dict of (value, bound) of dx (in dtype), dweight and dbias (in param)."""
    x, dout, n, dim = x.double(), dout.double(), *x.shape
    w = torch.ones(dim, dtype=torch.float64) if weight is None else weight.double()
    rstd = rstd.double()[:, None]
    h = (x - mean.double()[:, None]) * rstd
    g = dout * w
    sg, sgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = rstd * (g - sg - h * sgh)
    # h in two roundings, g in one, their product in one
    e_sg = (NORM_STEPS + 1) * U32 * g.abs().mean(1, keepdim=True)
    e_sgh = (NORM_STEPS + 4) * U32 * (g * h).abs().mean(1, keepdim=True)
    e_dx = rstd * (e_sg + h.abs() * e_sgh + 5 * U32 * (g.abs() + sg.abs() + (h * sgh).abs()))
    size, dw = (dout * h).abs().sum(0), (dout * h).sum(0)
    bsize, db = dout.abs().sum(0), dout.sum(0)
    return dict(dx=(dx, e_dx * (1 + u(dtype)) + u(dtype) * dx.abs() + tiny(dtype)),
                dweight=(dw, (n + 4) * U32 * size + u(param) * dw.abs() + tiny(param)),
                dbias=(db, (n + 1) * U32 * bsize + u(param) * db.abs() + tiny(param)))


# ---------------------------------------------------------------- losses


def _targets(rows, labels=None, ids=None, teacher=None, scale=1.0, pad=-1):
    """(live [n], target [n, rows], the teacher's part of the losses [n])"""
    if labels is not None:
        live = (labels >= 0) & (labels < rows) & (labels != pad)
        t = torch.zeros(len(labels), rows, dtype=torch.float64)
        t[live, labels[live]] = 1
        return live, t, torch.zeros(len(labels), dtype=torch.float64)
    on = (ids >= 0) & (ids < rows) & (ids != pad) & (teacher != -math.inf)
    live = on.any(1)
    s = (teacher.double() * scale).masked_fill(~on, -math.inf)
    q = torch.softmax(s.masked_fill(~live[:, None], 0.0), 1).masked_fill(~on, 0.0)
    t = torch.zeros(len(ids), rows, dtype=torch.float64)
    t.scatter_add_(1, torch.where(on, ids, 0), q)
    own = torch.where(q > 0, q * q.clamp_min(1e-300).log(), 0.0).sum(1)
    return live, t, own


def _scores(x, w, scale, live):
    """Scores of the tokens that take part (zeros for others) and their errors: dim
    fp32 multiply-adds and the scale."""
    x = torch.where(live[:, None], x.double(), 0.0)
    z = x @ w.double().T * scale
    size = abs(scale) * (x.abs() @ w.double().abs().T)
    return z, (x.shape[1] + 4) * U32 * size


def losses(x, w, scale=1.0, pad=-1, labels=None, ids=None, teacher=None):
    """dict of (value, bound) of loss and lse, and of logits with a teacher."""
    rows = w.shape[0]
    live, t, own = _targets(rows, labels, ids, teacher, scale, pad)
    z, e_z = _scores(x, w, scale, live)
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    big = z.abs().amax(1) + lse.abs()
    # the exponents' arguments and both logarithms in a few roundings; a sum of a
    # tile's scores, of a wave's and of the tiles
    e_lse = (p * e_z).sum(1) * 1.01 + 10 * U32 * big + (rows / 256 + 100) * U32
    e_loss = e_lse + (t * e_z).sum(1) + 16 * U32 * big
    if ids is not None:  # the teacher's softmax: arguments, exp, a sum of at most 256, log
        s = (teacher.double() * scale).abs().masked_fill(teacher == -math.inf, 0.0).amax(1)
        e_q = (8 * s + 280) * U32
        e_loss = e_loss + e_q * (1 + 2 * big + 2 * s) + ids.shape[1] * U32 * (big + s + own.abs())
    zero = torch.zeros_like(lse)
    res = dict(loss=(torch.where(live, own - (t * z).sum(1) + lse, zero), torch.where(live, e_loss, zero)),
               lse=(torch.where(live, lse, zero), torch.where(live, e_lse, zero)))
    if ids is not None:
        on = (ids >= 0) & (ids < rows) & (ids != pad) & (teacher != -math.inf)
        at = torch.where(on, ids, 0)
        res["logits"] = tuple(torch.where(on, y.gather(1, at), 0.0) for y in (z, e_z * 2 + 1e-40))
    return res


def loss_gradients(x, w, lse, dloss, dtype, scale=1.0, pad=-1, labels=None, ids=None, teacher=None):
    """dict of (value, bound) of dx (in x's type) and dweight (in dtype)."""
    rows, n, t = w.shape[0], x.shape[0], x.dtype
    live, target, _ = _targets(rows, labels, ids, teacher, scale, pad)
    z, e_z = _scores(x, w, scale, live)
    lse = torch.where(live, lse.double(), 0.0)[:, None]
    c = torch.where(live, dloss.double() * scale, 0.0)[:, None]
    p = torch.exp(z - lse)
    e = c * (p - target)
    # p: its exponent's argument (the factor's logarithm in it) and exp2; the
    # difference and the factor in one rounding each
    log = torch.where(c == 0, 0.0, c.abs().clamp_min(1e-300).log().abs()) + 40
    off = c.abs() * (p * (2 * e_z + 6 * U32 * (z.abs() + lse.abs() + log) + 4 * U32) + 4 * U32 * (p + target))
    if ids is not None:
        s = (teacher.double() * scale).abs().masked_fill(teacher == -math.inf, 0.0).amax(1, keepdim=True)
        off = off + c.abs() * target * (16 * s + 2 * 280) * U32
    # up to 256 tokens e is two numbers: what the rounding left is rounded once more
    once = u(t) * u(t) if n <= 256 else u(t)
    e_e = off * (1 + u(t)) + once * e.abs()
    if t == torch.float16:  # half a step of what is rounded times 2^13 .. 2^14 over the largest
        e_e = e_e + live[:, None] * 2.0 ** -38 * c.abs().max()
    xd, wd = torch.where(live[:, None], x.double(), 0.0), w.double()
    dx, dw = e @ wd, e.T @ xd
    b_dx = e_e @ wd.abs() + (rows + 40) * U32 * (e.abs() @ wd.abs())
    b_dw = e_e.T @ xd.abs() + (n + 40) * U32 * (e.abs().T @ xd.abs())
    return dict(dx=(dx, b_dx * (1 + u(t)) + u(t) * dx.abs() + live[:, None] * tiny(t)),
                dweight=(dw, b_dw * (1 + u(dtype)) + u(dtype) * dw.abs() + tiny(dtype)))
