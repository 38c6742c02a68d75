"""How far a gradient of the losses over a vocabulary's table may be from differences of
the losses.

With t the way along a direction v, f(t) = sum_i dloss_i loss_i(t) is held to the slope
(4 D(1) - D(2)) / 3 of its central differences D(k) = (f(k) - f(-k)) / 2 k.

What the slope leaves out: with f = sum a_k t^k, D(k) = sum over odd j of a_j k^(j - 1), so
the slope is a_1 - 4 a_5 - 20 a_7 - .., in all at most sum |a_j| 2^(j - 1) / 3 over j = 5, 7, ..
A token's scores move by t a_v where x alone moves or the table alone does, and its loss is
log sum p_v e^(t a_v) and a part that is linear in t (p: the softmax at t = 0). With R the range
of the a_v, taken about its middle, and |t| <= r = pi / 2 R, every exponent is at most pi / 4 in
size, so every term lies within pi / 4 of the real axis' direction, between e^(-pi / 4) and
e^(pi / 4) in size; the sum's real part is at least cos(pi / 4) e^(-pi / 4) = 0.32, its size at
most 2.2, its angle at most pi / 4. The logarithm is at most 1.14 + 0.79 < 2 in size there, and
|a_j| <= 2 r^-j. The sum of 2 r^-j 2^(j - 1) / 3 over j = 5, 7, .. is 32 / 3 r^-5 / (1 - 4 / r^2).

The direction is the gradient's own signs: the slope is then as large as the sum of its
terms' sizes, and a gradient that is wrong by a part of its size is off by that part."""

import math

import torch

import plain_head as H
from plain_ops import U32

STEP = 2.0 ** -8


def inputs(kind, seed=0):
    """(x, table, targets, dloss) whose elements are multiples of STEP below 4 in size, so
    that both ends of a difference hold them exactly in fp16; some tokens take no part."""
    n, rows, dim, top = 24, 90, 32, 5
    g = torch.Generator().manual_seed(seed)

    def grid(t):
        return (t.clamp(-3.9, 3.9) / STEP).round() * STEP

    w = grid(torch.randn(rows, dim, generator=g) * 2 / math.sqrt(dim))
    ids = torch.randint(0, rows, (n, top), generator=g)
    x = grid(torch.randn(n, dim, generator=g) + 0.5 * w[ids[:, 0]])
    ids[3], ids[11] = -1, -1
    s = dict(labels=ids[:, 0]) if kind == "loss" else \
        dict(ids=ids, teacher=3 * torch.randn(n, top, generator=g))
    return x.half(), w.half(), s, (torch.rand(n, generator=g) + 0.5) / n


def direction(grad):
    return grad.cpu().sign().double() * STEP


def left_out(x, w, vx, vw, dloss):
    """What the slope along vx or vw (the other is None) leaves out of f's derivative."""
    a = vx.double() @ w.double().T if vw is None else x.double() @ vw.double().T
    r = math.pi / 2 / (a.amax(1) - a.amin(1)).clamp_min(1e-9)
    assert r.min() > 4
    return float((dloss.double().abs() * 32 / 3 * r ** -5 / (1 - 4 / r ** 2)).sum())


def slope(f):
    """The slope of f, and what an error of f(t) of at most f(t)[1] does to it."""
    at = {t: f(t) for t in (-2, -1, 1, 2)}
    value = (4 * (at[1][0] - at[-1][0]) / 2 - (at[2][0] - at[-2][0]) / 4) / 3
    return value, (2 * (at[1][1] + at[-1][1]) + (at[2][1] + at[-2][1]) / 4) / 3


def off(x, w, s, dloss, side, grad, size, v, losses):
    """How far the gradient's slope along v is from the losses', and how far it may be: size
    bounds the gradient's error, losses(x, w) are (losses, their errors)."""
    vx, vw = (v, None) if side == "x" else (None, v)

    def f(t):
        a = x if vx is None else (x.double() + t * vx).to(x.dtype)
        b = w if vw is None else (w.double() + t * vw).to(w.dtype)
        moved = (a.double() - x.double() if vw is None else b.double() - w.double())
        assert torch.equal(moved, t * v)  # exact at both ends
        loss, error = losses(a, b)
        return float((loss * dloss.double()).sum()), float((error * dloss.double().abs()).sum())

    want, rounding = slope(f)
    have = float((grad.cpu().double() * v).sum())
    own = float((size * v.abs()).sum())
    return abs(have - want), rounding + own + left_out(x, w, vx, vw, dloss) + 100 * U32 * abs(want)


def plain(s):
    def losses(x, w):
        return H.losses(x, w, **s)["loss"]
    return losses
