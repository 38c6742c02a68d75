"""Losses of tokens against a vocabulary's table at their ends."""

import math

import pytest
import torch

import head_differences as D
import plain_head as H
import plain_ops as P
from test_gpu_token_loss import BF16, F16, F32, KINDS, backward, forward, inputs

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- sharp distributions


@pytest.mark.parametrize("k", [4, 8, 16, 40, 400])
@pytest.mark.parametrize("n,rows", [(64, 300), (300, 700), (300, 66_000)])
@pytest.mark.parametrize("t", [BF16, F16])
def test_a_certain_token_s_loss(n, rows, k, t):
    """Tokens at k times their label's row: scores of some hundreds beside which nothing else
    counts. No loss is below 0, and its error is that of what stands beside the label: with
    d_v = z_v - z_label, loss = log sum exp d_v, where a score's own rounding is the same in the
    label's place and in the sum's."""
    x, w, s, dloss = inputs("loss", n, rows, 64, t, masked=0.0, seed=k)
    lab = s["labels"]
    x = (k * w[lab].float()).to(t)
    got = forward(x.cuda(), w.cuda(), s)
    with torch.device("cuda"):
        z, e_z = H._scores(x.cuda(), w.cuda(), 1.0, torch.ones(n, dtype=torch.bool))
        at = lab.cuda()[:, None]
        d = (z - z.gather(1, at)).scatter(1, at, -math.inf)  # of the others
        rest = torch.exp(d).sum(1)
        loss = torch.log1p(rest)
        p = torch.exp(d) / (1 + rest)[:, None]
        bound = 1.02 * (p * (e_z + e_z.gather(1, at))).sum(1)
        # the sums of a tile, a wave and the tiles, near 1; exponents' arguments, of which
        # |d| e^d is what counts; both logarithms
        bound += (rows / 256 + 116) * P.U32 + 8 * P.U32 * loss
    assert (got["loss"] >= 0).all(), got["loss"].min()
    P.check(got["loss"], (loss.cpu(), bound.cpu()), "loss")


# ---------------------------------------------------------------- the teacher's ends


def _ends(t):
    """Rows of a teacher's logits and rows that have the same distribution."""
    low, high, none = torch.finfo(t).min, torch.finfo(t).max, -math.inf
    return [([low, low, low], [0.0, 0.0, 0.0]), ([high, high, high], [0.0, 0.0, 0.0]),
            ([low, 1.0, 2.0], [-60000.0, 1.0, 2.0]), ([low, high, low], [-60000.0, 0.0, -60000.0]),
            ([high, high, low], [0.0, 0.0, -60000.0]), ([low, none, low], [0.0, none, 0.0]),
            ([low, none, none], [7.0, none, none])]


@pytest.mark.parametrize("n", [7, 2100])
@pytest.mark.parametrize("scale", [0.01, 0.5, 1.0, 2.0])
@pytest.mark.parametrize("t", [F32, BF16, F16])
def test_a_teacher_s_largest_and_lowest_logits(t, scale, n):
    """Masks of the type's lowest value, alone too, and logits whose product with the scale
    passes fp32: a softmax knows only differences, so rows of the same differences, or of ones
    that fp32's exponential has no value for, give the same bits."""
    x, w, _, dloss = inputs("distill", n, 150, 64)
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(0, 150, (n, 3), generator=g)
    ends = _ends(t)
    a, b = (torch.tensor([ends[i % 7][j] for i in range(n)]).to(t) for j in (0, 1))
    sa, sb = dict(ids=ids, teacher=a), dict(ids=ids, teacher=b)
    got, want = (forward(x.cuda(), w.cuda(), s, scale=scale) for s in (sa, sb))
    for k in got:
        assert got[k].isfinite().all() and torch.equal(got[k], want[k]), k
    for y, z in zip(*(backward(x.cuda(), w.cuda(), s, want, dloss, scale=scale) for s in (sa, sb))):
        assert y.isfinite().all() and torch.equal(y, z)
    ref = H.losses(x, w, scale, **sb)
    for k, y in want.items():
        P.check(y, ref[k], k)


@pytest.mark.parametrize("t", [F32, BF16, F16])
def test_a_negative_scale_s_lowest_logit_is_certain(t):
    x, w, _, dloss = inputs("distill", 40, 150, 64)
    ids = torch.randint(0, 150, (40, 3), generator=torch.Generator().manual_seed(1))
    low = torch.tensor([[torch.finfo(t).min, 1.0, torch.finfo(t).max]]).repeat(40, 1).to(t)
    sure = torch.tensor([[-60000.0, 1.0, 60000.0]]).repeat(40, 1).to(t)
    got, want = (forward(x.cuda(), w.cuda(), dict(ids=ids, teacher=y), scale=-2.0) for y in (low, sure))
    for k in got:
        assert got[k].isfinite().all() and torch.equal(got[k], want[k]), k


# ---------------------------------------------------------------- differences


@pytest.mark.parametrize("side", ["x", "w"])
@pytest.mark.parametrize("kind", KINDS)
def test_gradients_against_differences(kind, side):
    """The calls' gradients against differences of the calls' own losses; test_head_differences
    has which wrong gradients these bounds refuse."""
    x, w, s, dloss = D.inputs(kind)
    got = forward(x.cuda(), w.cuda(), s)
    dx, dw = backward(x.cuda(), w.cuda(), s, got, dloss, dtype=F32)
    lse = got["lse"].cpu()
    ref = H.loss_gradients(x, w, lse, dloss, F32, **s)

    def losses(a, b):
        return forward(a.cuda(), b.cuda(), s)["loss"].cpu().double(), H.losses(a, b, **s)["loss"][1]

    grad, name = (dx, "dx") if side == "x" else (dw, "dweight")
    apart, most = D.off(x, w, s, dloss, side, grad, ref[name][1], D.direction(ref[name][0]), losses)
    assert apart <= most, (apart, most)
