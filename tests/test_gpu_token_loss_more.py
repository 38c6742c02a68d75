"""Losses of tokens against a vocabulary's table at their ends."""

import math

import pytest
import torch

import plain_head as H
import plain_ops as P
from test_gpu_token_loss import BF16, F16, forward, inputs

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
