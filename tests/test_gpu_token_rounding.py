"""The token gradient is the 64-bit sum rounded once: sums a little beside a
midpoint of the 16-bit types, which rounding to fp32 on the way would put on it."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BITS = {torch.bfloat16: 8, torch.float16: 11}  # of a value, the leading one among them


@pytest.fixture(scope="module")
def L():
    from jagged_embedding_sparse_amd import lib
    return lib


def _once(x, dtype):
    """x (64 bits, in the type's normal range) to the nearest value, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs())) - (BITS[dtype] - 1))
    return (torch.round(x / step) * step).to(dtype)


def _parts(dtype, dim):
    """Three fp32 numbers per column whose sum is beside a midpoint, and the sum:
    a value of the type, half its step, and 2^-26 .. 2^-45 of it either way or 0."""
    c = torch.arange(dim, dtype=torch.float64)
    value = (1 + (c % 64) / 64) * torch.exp2(c % 13 - 6)
    unit = torch.exp2(torch.floor(torch.log2(value)))
    half = unit * 2.0 ** -BITS[dtype]
    rest = unit * torch.exp2(-26 - c % 20) * (c % 3 - 1)
    sign = 1 - 2 * (c // 7 % 2)
    parts = torch.stack([value, half, rest]) * sign
    assert (parts.float().double() == parts).all()
    return parts.float(), parts.sum(0)


def test_the_plain_rounding():
    for t in BITS:
        x = torch.randn(1000, generator=torch.Generator().manual_seed(1)).double()
        assert torch.equal(_once(x, t), x.to(t))  # fp32 values: one rounding in torch too


@pytest.mark.parametrize("dtype", list(BITS))
@pytest.mark.parametrize("dim", [1, 6, 264, 1003])
@pytest.mark.parametrize("lead", [0, 100, 3000])
def test_sums_beside_a_midpoint(L, dtype, dim, lead):
    """Rows summed whole, over chunks, and over workgroups (tokens of zeros
    before the three)."""
    parts, exact = _parts(dtype, dim)
    dout = torch.cat([torch.zeros(lead, dim), parts, torch.ones(4, dim)])
    ids = torch.cat([torch.full((lead + 3,), 2), torch.tensor([0, 1, 3, 4])])
    uq = L.fs_token_sort(ids.cuda(), 6)
    got = L.fs_token_grad(uq, dout.cuda(), 6, dtype=dtype).cpu()
    assert torch.equal(got[2], _once(exact, dtype))
    got = L.fs_token_grad(uq, dout.cuda(), 6, scale=-4.0, dtype=dtype).cpu()
    assert torch.equal(got[2], _once(-4 * exact, dtype))


@pytest.mark.parametrize("dtype", list(BITS))
def test_accumulated_beside_a_midpoint(L, dtype):
    parts, exact = _parts(dtype, 200)
    grad = parts[:1].to(dtype).cuda()
    assert torch.equal(grad.cpu().float(), parts[:1])
    uq = L.fs_token_sort(torch.zeros(2, dtype=torch.int64).cuda(), 1)
    L.fs_token_grad(uq, parts[1:].contiguous().cuda(), 1, grad=grad, accumulate=True)
    assert torch.equal(grad[0].cpu(), _once(exact, dtype))


@pytest.mark.parametrize("dtype", list(BITS) + [torch.float32])
def test_infinities_nan_and_the_ends_of_the_range(L, dtype):
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    dout = torch.tensor([[float("inf"), float("-inf"), float("nan"), big, -big, tiny, 0.0, -0.0]])
    uq = L.fs_token_sort(torch.zeros(1, dtype=torch.int64).cuda(), 1)
    got = L.fs_token_grad(uq, dout.cuda(), 1, dtype=dtype).cpu().float()
    assert torch.equal(got.nan_to_num(7.0, 9e38, -9e38), dout.nan_to_num(7.0, 9e38, -9e38))
    # fp32 values past the type's largest, and below half its smallest
    if dtype != torch.float32:
        half = torch.tensor([[big, big, tiny, tiny]])
        dout = torch.cat([half, torch.tensor([[big, big / 1024, -tiny / 2, -tiny * 0.5001]])])
        uq = L.fs_token_sort(torch.zeros(2, dtype=torch.int64).cuda(), 1)
        got = L.fs_token_grad(uq, dout.cuda(), 1, dtype=dtype).cpu().double()[0].tolist()
        # half a step at the largest value: fp16 16, bf16 2^119, of which the column has 2^118
        assert got[0] == float("inf")
        assert got[1] == (big if dtype == torch.bfloat16 else float("inf"))
        assert got[2] == 0.0 and got[3] == 0.0
