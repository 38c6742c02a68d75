"""The plain forms' own gradients against differences of their values, in 64 bits.

A central difference over steps of h = 2^-10 of two sizes, (4 D(h) - D(2 h)) / 3,
leaves out the third derivative: what remains is of the order h^4 = 2^-40 of the
terms, and the values' rounding over h, 2^-53 2^10. 1e-8 of the terms' sizes holds
both with derivatives of some hundreds."""

import math

import pytest
import torch

import plain_head as H

F64 = torch.float64
h = 2.0 ** -10


def slope(f, at, direction):
    d = [(f(at + k * h * direction) - f(at - k * h * direction)) / (2 * k * h) for k in (1, 2)]
    return (4 * d[0] - d[1]) / 3


def same(f, at, grad, seed=0):
    g = torch.Generator().manual_seed(seed)
    for _ in range(3):
        v = torch.randn(at.shape, generator=g, dtype=F64)
        size = float((grad * v).abs().sum()) + 1e-3
        assert abs(float(slope(f, at, v)) - float((grad * v).sum())) <= 1e-8 * size


@pytest.mark.parametrize("n,dim,affine", [(1, 5, True), (7, 12, True), (6, 33, False)])
def test_norm(n, dim, affine):
    g = torch.Generator().manual_seed(n)
    x, dout = (torch.randn(n, dim, generator=g, dtype=F64) for _ in range(2))
    w = 1 + 0.3 * torch.randn(dim, generator=g, dtype=F64) if affine else None
    b = torch.randn(dim, generator=g, dtype=F64) if affine else None

    def total(x, w, b):
        return (H.norm(x, w, b, 1e-3, F64)["out"][0] * dout).sum()

    y = H.norm(x, w, b, 1e-3, F64)
    grad = H.norm_backward(x, y["mean"][0], y["rstd"][0], dout, w, F64, F64)
    same(lambda t: total(t, w, b), x, grad["dx"][0])
    if affine:
        same(lambda t: total(x, t, b), w, grad["dweight"][0])
        same(lambda t: total(x, w, t), b, grad["dbias"][0])


@pytest.mark.parametrize("kind", ["loss", "distill"])
@pytest.mark.parametrize("scale", [1.0, -0.7])
def test_losses(kind, scale):
    g = torch.Generator().manual_seed(5)
    n, rows, dim, top = 9, 23, 6, 4
    x, w = (torch.randn(m, dim, generator=g, dtype=F64) for m in (n, rows))
    dloss = torch.rand(n, generator=g, dtype=F64)
    if kind == "loss":
        s = dict(labels=torch.randint(0, rows, (n,), generator=g))
        s["labels"][2:4] = torch.tensor([-1, rows])
    else:
        s = dict(ids=torch.randint(0, rows, (n, top), generator=g),
                 teacher=torch.randn(n, top, generator=g, dtype=F64))
        s["ids"][3] = -1            # takes no part
        s["ids"][4, 1:] = rows + 1  # one entry
        s["ids"][5] = 7             # one id in every entry
        s["teacher"][6, 0] = -math.inf

    def total(x, w):
        return (H.losses(x, w, scale, **s)["loss"][0] * dloss).sum()

    lse = H.losses(x, w, scale, **s)["lse"][0]
    grad = H.loss_gradients(x, w, lse, dloss, F64, scale, **s)
    same(lambda t: total(t, w), x, grad["dx"][0])
    same(lambda t: total(x, t), w, grad["dweight"][0])
    assert not grad["dx"][0][3].any()


def test_a_loss_of_one_certain_entry_is_the_label_s():
    g = torch.Generator().manual_seed(6)
    x, w = (torch.randn(m, 4, generator=g, dtype=F64) for m in (5, 11))
    ids = torch.randint(0, 11, (5, 1), generator=g)
    a = H.losses(x, w, labels=ids[:, 0])
    b = H.losses(x, w, ids=ids, teacher=torch.randn(5, 1, generator=g, dtype=F64))
    assert torch.allclose(a["loss"][0], b["loss"][0], rtol=0, atol=1e-12)
    assert torch.allclose(
        a["loss"][0], -torch.log_softmax(x @ w.T, 1).gather(1, ids)[:, 0], rtol=0, atol=1e-12)
