"""Differences of the losses tell a right gradient from wrong ones: the plain form's
passes, and each of a list of mistakes fails, with the bounds that the kernels' gradients
are held to."""

import pytest
import torch

import head_differences as D
import plain_head as H

MISTAKES = dict(
    ten_times=lambda g, *_: 10 * g, half=lambda g, *_: g / 2, five_percent=lambda g, *_: 1.05 * g,
    negated=lambda g, *_: -g, without_the_target=lambda g, p, t: p, target_alone=lambda g, p, t: t,
    rows_shuffled=lambda g, *_: g.roll(1, 0), nothing=lambda g, *_: 0 * g)


def gradients(kind):
    """For x and for the table: (gradient, its error's bound, its softmax part, its target part)"""
    x, w, s, dloss = D.inputs(kind)
    lse = H.losses(x, w, **s)["lse"][0]
    ref = H.loss_gradients(x, w, lse, dloss, torch.float16, **s)
    live, target, _ = H._targets(w.shape[0], **s)
    t = -torch.where(live[:, None], dloss.double()[:, None], 0.0) * target
    xd = torch.where(live[:, None], x.double(), 0.0)
    parts = dict(x=(ref["dx"], t @ w.double()), w=(ref["dweight"], t.T @ xd))
    return (x, w, s, dloss), {k: (v, size, v - at, at) for k, ((v, size), at) in parts.items()}


@pytest.mark.parametrize("side", ["x", "w"])
@pytest.mark.parametrize("kind", ["loss", "distill"])
def test_the_right_gradient_passes(kind, side):
    given, parts = gradients(kind)
    grad, size, *_ = parts[side]
    apart, most = D.off(*given, side, grad, size, D.direction(grad), D.plain(given[2]))
    assert apart <= most


@pytest.mark.parametrize("mistake", list(MISTAKES))
@pytest.mark.parametrize("side", ["x", "w"])
@pytest.mark.parametrize("kind", ["loss", "distill"])
def test_a_wrong_gradient_fails(kind, side, mistake):
    given, parts = gradients(kind)
    grad, size, softmax, target = parts[side]
    wrong = MISTAKES[mistake](grad, softmax, target)
    apart, most = D.off(*given, side, wrong, size, D.direction(grad), D.plain(given[2]))
    assert apart > most
