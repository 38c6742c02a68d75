"""Layer norm where its sums are exact: a sum over a row is divided by the row's length in one
rounding, so what the formula says is nothing is nothing."""

import pytest
import torch

from jagged_embedding_sparse_amd import lib as L

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16

# one width for every number of lanes and pieces that a row is shared by, and a few more
WIDTHS = [1, 3, 7, 10, 29, 41, 48, 93, 100, 130, 250, 300, 500, 700, 1000, 1500, 2000, 2100, 2900, 3500,
          4000, 4200, 5000, 6200, 7000, 8000, 8300, 10000, 12000, 13000, 16000]


@pytest.mark.parametrize("x", [F32, BF16, F16])
@pytest.mark.parametrize("dim", WIDTHS)
def test_rows_of_one_number(dim, x):
    """Whole numbers whose sums fp32 holds: their mean is the number, nothing is left of the
    centred row, and the output is the bias."""
    at = torch.tensor([3.0, -5.0, 7.0, 11.0, 100.0, 1000.0, 0.0])
    rows = at[:, None].repeat(1, dim).to(x).cuda()
    bias = torch.arange(dim, device="cuda") / 64.0
    out, mean, rstd = L.fs_layer_norm(rows, torch.full((dim,), 1.5, device="cuda"), bias, eps=1e-6, dtype=F32)
    assert torch.equal(mean.cpu(), at)
    assert torch.equal(out, bias.expand(7, dim))
    assert (rstd == rstd[0]).all()


@pytest.mark.parametrize("n", [3, 40, 3000])
@pytest.mark.parametrize("x", [F32, BF16])
@pytest.mark.parametrize("dim", WIDTHS)
def test_a_gradient_along_the_mean_is_nothing(dim, x, n):
    """The output does not change with a row's mean: dout of one whole number, without a
    weight, gives dx = 0 where the h of a row add up to 0."""
    h = torch.ones(dim)
    h[1::2] = -1
    if dim % 2:
        h[-1] = 0
    at = torch.tensor([3.0, -5.0, 7.0, 11.0, 25.0])
    dout = at[torch.arange(n) % 5][:, None].repeat(1, dim).to(x).cuda()
    dx, _, _ = L.fs_layer_norm_backward(h.repeat(n, 1).to(x).cuda(), torch.zeros(n, device="cuda"),
                                        torch.ones(n, device="cuda"), dout)
    assert not dx.any()
