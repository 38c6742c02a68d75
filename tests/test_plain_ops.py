"""The plain 64-bit forms that the GPU tests compare with, by hand examples,
by torch's own gradients and by differences."""

import math

import torch

import plain_ops as P


def _inputs(lens, hq, hk, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    off = [0]
    for x in lens:
        off.append(off[-1] + x)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(n, hq, d), r(n, hk, d), r(n, hk, d), r(n, hq, d), off


def test_mask_by_hand():
    # two history tokens, two candidates: the candidates see the history and themselves
    want = torch.tensor([[1, 0, 0, 0], [1, 1, 0, 0], [1, 1, 1, 0], [1, 1, 0, 1]]).bool()
    assert torch.equal(P.sees(4, 2, True), want)
    want[0, 1] = True
    assert torch.equal(P.sees(4, 2, False), want)
    assert torch.equal(P.sees(3, 3, True), torch.eye(3).bool())
    assert not P.sees(2, 0, True, torch.tensor([False, True]))[:, 0].any()


def test_one_token_and_empty_row():
    q, k, v, _, off = _inputs([1, 2], 2, 1, 8)
    res = P.attention(q, k, v, off, None, torch.tensor([1, 0, 0]), True, 0.3)
    assert torch.allclose(res["out"][0][0], v[0].expand(2, 8))
    assert torch.allclose(res["lse"][0][:, 0], 0.3 * (q[0] * k[0]).sum(1))
    assert (res["out"][0][1:] == 0).all() and (res["lse"][0][:, 1:] == -math.inf).all()


def _loss(q, k, v, do, off, cand, valid, causal, scale):
    return (P.attention(q, k, v, off, cand, valid, causal, scale)["out"][0] * do).sum()


def test_attention_gradient_by_autograd_and_differences():
    for causal in (True, False):
        q, k, v, do, off = _inputs([5, 1, 9], 4, 2, 8, seed=int(causal))
        cand, valid = torch.tensor([2, 0, 9]), torch.ones(15, dtype=torch.uint8)
        valid[3] = 0
        args = (off, cand, valid, causal, 0.4)
        got = P.attention(q, k, v, *args, dout=do)
        for x in (q, k, v):
            x.requires_grad_()
        ref = torch.autograd.grad(_loss(q, k, v, do, *args), (q, k, v))
        for name, r in zip(("dq", "dk", "dv"), ref):
            assert torch.allclose(got[name][0], r, atol=1e-12), name
        with torch.no_grad():
            eps = 1e-5
            for x, name in ((q, "dq"), (k, "dk"), (v, "dv")):
                step = torch.randn(x.shape, dtype=torch.float64,
                                   generator=torch.Generator().manual_seed(7))
                x += eps * step
                up = _loss(q, k, v, do, *args)
                x -= 2 * eps * step
                down = _loss(q, k, v, do, *args)
                x += eps * step
                slope = (got[name][0] * step).sum()
                assert abs((up - down) / (2 * eps) - slope) < 1e-7 * (1 + abs(slope)), name


def test_token_forms_by_hand_and_differences():
    ids = torch.tensor([3, 0, 3, -1, 7, 1, 3])
    assert P.token_sort(ids, 5, 1) == ([0, 3], [0, 1, 4], [1, 0, 2, 6], [0, 1, 1, 1])
    g = torch.Generator().manual_seed(1)
    w = torch.randn(5, 3, generator=g, dtype=torch.float64)
    do = torch.randn(7, 3, generator=g, dtype=torch.float64)
    out = P.token_lookup(w, ids, 2.0)
    assert torch.equal(out[0], 2 * w[3]) and (out[3:5] == 0).all()
    grad, _ = P.token_grad(ids, do, 5, -1, 2.0)
    step = torch.randn(5, 3, generator=g, dtype=torch.float64)
    up, down = ((P.token_lookup(w + s * step, ids, 2.0) * do).sum() for s in (1e-4, -1e-4))
    assert abs((up - down) / 2e-4 - (grad * step).sum()) < 1e-9
    assert (P.token_grad(ids, do, 5, 3, 2.0)[0][3] == 0).all()  # the padding row
