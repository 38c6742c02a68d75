"""Rows that see themselves alone: their softmax is 1 whatever their score is, so
nothing of them reaches dq and dk, to the bit, and dv is dout."""

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def L():
    from jagged_embedding_sparse_amd import lib
    return lib


def _run(L, lens, hq, hk, d, t, causal=True, cand=None, valid=None, spread=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    off = torch.tensor([0] + lens).cumsum(0).cuda()
    r = lambda h: (torch.randn(n, h, d, generator=g) * spread).to(t).cuda()  # noqa: E731
    q, k, v, do = r(hq), r(hk), r(hk), r(hq)
    kw = dict(n_cand=None if cand is None else torch.tensor(cand, dtype=torch.int32).cuda(),
              valid=None if valid is None else valid.cuda(), causal=causal)
    out, lse = L.fs_jagged_attention(q, k, v, off, **kw)
    dq, dk, dv = L.fs_jagged_attention_backward(q, k, v, out, lse, do, off, **kw)
    return q, k, v, do, out, dq, dk, dv


def _check(alone, group, v, do, out, dq, dk, dv):
    assert torch.equal(out[alone], v.repeat_interleave(group, 1)[alone])
    assert (dq[alone] == 0).all()
    return dk, dv


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d", [8, 32, 40, 64, 96, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("spread", [0.1, 1.0, 6.0])
def test_samples_of_one_token(L, t, d, causal, spread):
    lens = [1, 0, 1, 1] * 50
    _, _, v, do, out, dq, dk, dv = _run(L, lens, 2, 2, d, t, causal, spread=spread, seed=d)
    _check(slice(None), 1, v, do, out, dq, dk, dv)
    assert (dk == 0).all() and torch.equal(dv, do)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 2), (8, 2)])
def test_candidates_without_a_history(L, t, d, hq, hk):
    """Samples of candidates alone, over one and several tiles."""
    lens = [1, 33, 64, 130, 300]
    _, _, v, do, out, dq, dk, dv = _run(L, lens, hq, hk, d, t, cand=lens, seed=d)
    _check(slice(None), hq // hk, v, do, out, dq, dk, dv)
    assert (dk == 0).all()
    want = do.double().unflatten(1, (hk, -1)).sum(2)
    eps = torch.finfo(t).eps  # P and the result: half a step each
    assert ((dv.double() - want).abs() <= eps * do.double().abs().unflatten(1, (hk, -1)).sum(2)).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d", [32, 64, 128])
def test_first_rows_and_rows_behind_tokens_that_take_no_part(L, t, d):
    """A causal sample's first live row, wherever it is in the first tiles, and
    candidates behind a history of which nothing takes part."""
    lens, cand = [100, 90, 128, 70], [0, 0, 0, 9]
    valid = torch.ones(sum(lens), dtype=torch.uint8)
    valid[100:140] = 0  # sample 1: its row 40 is the first
    valid[190:253] = 0  # sample 2: its row 63
    valid[318:379] = 0  # sample 3: candidates alone
    q, k, v, do, out, dq, dk, dv = _run(L, lens, 2, 1, d, t, cand=cand, valid=valid, seed=d)
    alone = torch.tensor([0, 140, 253] + list(range(379, 388)))
    _check(alone, 2, v, do, out, dq, dk, dv)
    assert (dk[379:388] == 0).all()
    for y in (out, dq, dk, dv):
        assert y.isfinite().all() and (y.cpu()[valid == 0] == 0).all()
    assert (dq[1:100] != 0).any(2).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d", [24, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_one_live_token_of_a_long_sample(L, t, d, causal):
    """Rows of many steps that see themselves alone: one live token, and
    candidates behind a long history of which nothing takes part."""
    lens, cand = [1000, 800], [0, 70]
    valid = torch.zeros(sum(lens), dtype=torch.uint8)
    alone = torch.tensor([700] + list(range(1730, 1800)))
    valid[alone] = 1
    q, k, v, do, out, dq, dk, dv = _run(L, lens, 4, 1, d, t, causal, cand, valid, seed=d)
    _check(alone, 4, v, do, out, dq, dk, dv)
    assert (dk == 0).all()
    for y in (out, dq, dk, dv):
        assert y.isfinite().all() and (y.cpu()[valid == 0] == 0).all()
