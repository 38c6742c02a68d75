"""Plain 64-bit forms of the layer norm and of the losses over a vocabulary's
table, on the CPU, and how far a result rounded to fewer bits may be from them
(plain_ops has how bounds count roundings)."""

import math

import torch

from plain_ops import U32, tiny, u

# A row's sum in the kernels: at most 16 values of a lane, 6 exchanges inside a
# wave, at most 16 waves, and the division by dim.
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
