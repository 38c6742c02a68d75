"""Layer norm where its sums are exact (a sum over a row is divided by the row's length in one
rounding, so what the formula says is nothing is nothing), at every width with types mixed, and
at sizes past 32 bits."""

import math

import pytest
import torch

import plain_head as H
import plain_ops as P
from jagged_embedding_sparse_amd import lib as L
from test_gpu_norm import _both, _inputs

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


@pytest.mark.parametrize("n", [2, 37, 700])
@pytest.mark.parametrize("x,out,param", [(F32, BF16, F16), (F16, F32, BF16)])
@pytest.mark.parametrize("dim", WIDTHS)
def test_mixed_types_at_every_width(dim, x, out, param, n):
    _both(n, dim, x, out, param, seed=n)


def test_eps_of_nothing():
    _both(40, 100, F32, F32, eps=0.0)


@pytest.mark.parametrize("which", ["dweight", "dbias"])
@pytest.mark.parametrize("n", [3, 4000])
def test_one_parameter_s_gradient_alone(n, which):
    xs, _, _, dout = _inputs(n, 72)
    _, mean, rstd = L.fs_layer_norm(xs.cuda())
    y = torch.full((72,), math.nan, device="cuda")
    _, *both = L.fs_layer_norm_backward(xs.cuda(), mean, rstd, dout.cuda(), **{which: y})
    assert both[which == "dweight"] is None
    P.check(y, H.norm_backward(xs, mean.cpu(), rstd.cpu(), dout, None, F32, F32)[which], which)


@pytest.mark.parametrize("keep", [(True, False), (False, True), (False, False)])
def test_the_c_call_without_statistics(keep):
    xs, w, b, _ = (t.cuda() for t in _inputs(50, 200))
    want = L.fs_layer_norm(xs, w, b)
    out = torch.full_like(xs, math.nan)
    stats = [torch.full((50,), math.nan, device="cuda") for _ in range(2)]
    rc = L._c_layer_norm(xs.data_ptr(), L.FS_F32, 0, 50, 200, w.data_ptr(), b.data_ptr(), L.FS_F32, 1e-5,
                         out.data_ptr(), L.FS_F32, 0, *(t.data_ptr() if k else None for t, k in zip(stats, keep)),
                         torch.cuda.current_stream().cuda_stream)
    assert rc == L.FS_OK and torch.equal(out, want[0])
    for t, k, y in zip(stats, keep, want[1:]):
        assert torch.equal(t, y) if k else t.isnan().all()


def test_rows_past_32_bits():
    """4.5 GB each of x, out, dout and dx."""
    n, dim, step = 1_100_000, 1024, 100_000
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dout = (torch.empty(n, dim, device="cuda").normal_(generator=g) for _ in range(2))
    w, b = (torch.empty(dim, device="cuda").normal_(generator=g) for _ in range(2))
    out, mean, rstd = L.fs_layer_norm(x, w, b)
    dx, dw, db = L.fs_layer_norm_backward(x, mean, rstd, dout, w)
    sums = {}
    with torch.device("cuda"):
        for lo in range(0, n, step):
            at = slice(lo, lo + step)
            ref = H.norm(x[at], w, b, 1e-5, F32)
            for name, y in (("out", out), ("mean", mean), ("rstd", rstd)):
                assert ((y[at].double() - ref[name][0]).abs() <= ref[name][1]).all(), (name, lo)
            ref = H.norm_backward(x[at], mean[at], rstd[at], dout[at], w, F32, F32)
            assert ((dx[at].double() - ref["dx"][0]).abs() <= ref["dx"][1]).all(), lo
            # sums of 1024 workgroups' rows, a workgroup's groups and the workgroups' sums
            h = (x[at].double() - mean[at, None].double()) * rstd[at, None].double()
            for name, terms in (("dweight", dout[at] * h), ("dbias", dout[at].double())):
                v, size = sums.get(name, (0, 0))
                sums[name] = (v + terms.sum(0), size + terms.abs().sum(0))
    for name, y in (("dweight", dw), ("dbias", db)):
        v, size = sums[name]
        P.check(y, (v.cpu(), ((n / 768 + 1024 + 8) * P.U32 * size).cpu()), name)


def test_the_most_rows():
    """2^31 - 2 rows of one column: each is its own mean."""
    n, step = (1 << 31) - 2, 1 << 28
    x = torch.empty(n, 1, dtype=BF16, device="cuda")
    for lo in range(0, n, step):
        x[lo:lo + step] = (torch.arange(min(step, n - lo), device="cuda") % 253 - 100)[:, None].to(BF16)
    w, b = (torch.full((1,), v, dtype=BF16, device="cuda") for v in (1.5, 0.25))
    out, mean, rstd = L.fs_layer_norm(x, w, b, eps=1.0)
    for lo in range(0, n, step):
        at = slice(lo, lo + step)
        assert (out[at] == 0.25).all() and torch.equal(mean[at], x[at, 0].float()) and (rstd[at] == 1).all()
    dx, dw, db = L.fs_layer_norm_backward(x, mean, rstd, out, w)
    assert not any(dx[lo:lo + step].any() for lo in range(0, n, step)) and float(dw) == 0
    # groups of 8 lanes add 2^16 rows of 0.25, exactly; 2^15 of them, and every sum is a
    # multiple of 2^14 below 2^29 but the last rows', so it is exact until bf16's rounding
    assert abs(float(db) - n / 4) <= P.u(BF16) * n / 4
