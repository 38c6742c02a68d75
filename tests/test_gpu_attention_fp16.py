"""The attention in fp16 where P and dS leave fp16's range and the inputs and
outputs do not: long samples, small gradients, gradients scaled up against
underflow. Against 64 bits, with bounds that allow a result its own rounding
and P and dS half a step each, which ends only far below the largest of them."""

import math

import pytest
import torch

import plain_ops as P

pytestmark = pytest.mark.gpu

HF = torch.float16
UT, U32, TINY = P.u(HF), P.U32, P.tiny(HF)


@pytest.fixture(scope="module")
def L():
    from jagged_embedding_sparse_amd import lib
    return lib


class Case:
    """Spreads of q, k, v and dout; rows(i) scales dout's row i of a sample of
    its length, keys(j) likewise v's."""

    def __init__(self, lens, hq, hk, d, causal, cand=None, masked=0.0, q=1.0, k=1.0, v=1.0, do=1.0,
                 scale=None, rows=None, keys=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        n = sum(lens)
        self.off = torch.tensor([0] + lens).cumsum(0)
        self.lens, self.hq, self.hk, self.d, self.causal = lens, hq, hk, d, causal
        self.cand = [0] * len(lens) if cand is None else cand
        self.scale = d ** -0.5 if scale is None else scale
        at = torch.cat([torch.arange(x) / max(x - 1, 1) for x in lens])[:, None, None]
        r = lambda h, s: torch.randn(n, h, d, generator=g) * s  # noqa: E731
        self.q, self.k, self.v, self.do = r(hq, q), r(hk, k), r(hk, v), r(hq, do)
        if rows:
            self.do = self.do * rows(at)
        if keys:
            self.v = self.v * keys(at)
        self.q, self.k, self.v, self.do = (x.to(HF) for x in (self.q, self.k, self.v, self.do))
        self.valid = None
        if masked:
            self.valid = (torch.rand(n, generator=g) >= masked).to(torch.uint8)

    def run(self, L):
        up = lambda x: None if x is None else x.cuda()  # noqa: E731
        kw = dict(n_cand=torch.tensor(self.cand, dtype=torch.int32).cuda(), valid=up(self.valid),
                  causal=self.causal, scale=self.scale)
        q, k, v, off = up(self.q), up(self.k), up(self.v), up(self.off)
        out, lse = L.fs_jagged_attention(q, k, v, off, **kw)
        dq, dk, dv = L.fs_jagged_attention_backward(q, k, v, out, lse, up(self.do), off, **kw)
        got = dict(dq=dq, dk=dk, dv=dv)
        for s in range(len(self.lens)):
            lo, hi = int(self.off[s]), int(self.off[s + 1])
            if lo < hi:
                for name, ref in self.ref(s, lo, hi, out[lo:hi].cpu()).items():
                    P.check(got[name][lo:hi].permute(1, 0, 2), ref, f"{name} of sample {s}")

    def ref(self, s, lo, hi, out16):
        """(value, bound) of one sample, heads first."""
        n, group = hi - lo, self.hq // self.hk
        ok = torch.ones(n, dtype=torch.bool) if self.valid is None else self.valid[lo:hi] != 0
        see = P.sees(n, self.cand[s], self.causal, ok)
        mine = lambda x, rep: torch.where(ok[:, None, None], x[lo:hi].double(), 0.0).permute(  # noqa: E731
            1, 0, 2).repeat_interleave(rep, 0)
        q, k, v, do = mine(self.q, 1), mine(self.k, group), mine(self.v, group), mine(self.do, 1)
        a = (q @ k.mT * self.scale).masked_fill(~see, -math.inf)
        lse = torch.logsumexp(a, 2)
        p = torch.exp(a - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
        # fp32: S (d steps), the exponent's argument and lse, exp2, the sums over keys
        size = torch.where(see, abs(self.scale) * (q.abs() @ k.abs().mT), 0.0).amax((1, 2), True)
        rel = ((self.d + 4) * size + 4 * lse.abs().masked_fill(torch.isinf(lse), 0.0).amax() + 24
               + 4 * math.log2(n + 1) + n) * U32
        res = {}
        o = p @ v
        # backward, from the out that the forward call stored: its error is what
        # delta has beside fp32's
        o16 = out16.double().permute(1, 0, 2)
        dp, dsize = do @ v.mT, do.abs() @ v.abs().mT
        delta = (do * o).sum(2, keepdim=True)
        d_size = (do * o).abs().sum(2, keepdim=True)
        off_delta = (do * (o16 - o)).abs().sum(2, keepdim=True)
        ds = p * (dp - delta)
        fp32 = 2 * rel * ds.abs() + p * ((self.d + 4) * U32 * (dsize + d_size) + off_delta)
        # the largest dS of the row, and of the rows that meet the key's tile
        row_top = ds.abs().amax(2, keepdim=True)
        tops = row_top.reshape(self.hk, group, n).amax(1)
        if self.causal:
            tops = tops.flip(1).cummax(1).values.flip(1)
            tops = tops[:, torch.arange(n) // 128 * 128]
        else:
            tops = tops.amax(1, keepdim=True).expand(-1, n)
        tops = tops.repeat_interleave(group, 0)[:, None, :]
        zero = 2.0 ** -24 * (p * d_size)  # dS that cancel are rounding errors of delta
        e_q = UT * ds.abs() + fp32 + see * 2.0 ** -36 * row_top + zero
        e_k = UT * ds.abs() + fp32 + see * 2.0 ** -34 * tops + zero
        e_v = (UT + 2 * rel) * p + see * 2.0 ** -37

        def shared(x):
            return x.reshape(self.hk, group, n, self.d).sum(1)

        n32 = (n * group + 8) * U32
        dq = ds @ k * self.scale
        b = e_q @ k.abs() + n32 * (ds.abs() @ k.abs())
        res["dq"] = (dq, b * abs(self.scale) + UT * dq.abs() + TINY)
        dk = shared(ds.mT @ q) * self.scale
        b = shared(e_k.mT @ q.abs() + n32 * (ds.abs().mT @ q.abs()))
        res["dk"] = (dk, b * abs(self.scale) + UT * dk.abs() + TINY)
        dv = shared(p.mT @ do)
        b = shared(e_v.mT @ do.abs() + n32 * (p.mT @ do.abs()))
        res["dv"] = (dv, b + UT * dv.abs() + TINY)
        return res


@pytest.mark.parametrize("d,hq,hk", [(64, 2, 1), (128, 2, 2), (40, 4, 1), (32, 1, 1)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("side", ["q", "k"])
def test_small_gradients_of_long_samples(L, d, hq, hk, causal, side):
    """Gradients of 1e-4 over 2100 tokens: dS is about 1e-7, fp16's smallest
    step 6e-8. One of q and k is large, so that dk or dq stays in range."""
    big = {"q": 16.0 if side == "q" else 1 / 16, "k": 16.0 if side == "k" else 1 / 16}
    Case([2100, 3], hq, hk, d, causal, do=1e-4, seed=d, **big).run(L)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_gradients_scaled_up(L, d, causal):
    """dS of several times fp16's largest value, with dq, dk and dv inside it."""
    Case([2, 40, 300], 2, 1, d, causal, v=8.0, do=2000.0, scale=0.01, q=3.0, k=3.0, seed=d).run(L)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_and_keys_of_very_different_sizes(L, d, causal):
    """Gradients that fall or rise by 2^20 along the sample, values that rise
    along it: a row's factor moves while it passes over the keys."""
    for i, (rows, keys) in enumerate([(lambda x: 2.0 ** (-20 * x), None), (lambda x: 2.0 ** (20 * x - 20), None),
                                      (None, lambda x: 2.0 ** (20 * x - 12)),
                                      (None, lambda x: 2.0 ** (8 - 20 * x))]):
        Case([700, 130], 4, 2, d, causal, rows=rows, keys=keys, k=4.0, q=0.5, seed=i).run(L)


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_with_a_gradient(L, d):
    """Candidates alone have a gradient, in one sample nobody has, and tokens
    take no part: rows and whole tiles without a factor."""
    c = Case([600, 300, 129], 2, 1, d, True, cand=[5, 0, 129], masked=0.2, do=1e-4, k=16.0, q=1 / 16)
    c.do[:595] = 0
    c.do[600:900] = 0
    c.run(L)


def test_infinities_and_nan_stay_in_their_sample(L):
    c = Case([70, 300, 70], 2, 2, 64, True, seed=2)
    clean = [x.cuda() for x in (c.q, c.k, c.v, c.do)]
    off = c.off.cuda()
    out, lse = L.fs_jagged_attention(*clean[:3], off)
    want = L.fs_jagged_attention_backward(*clean[:3], out, lse, clean[3], off)
    for bad in (math.nan, math.inf):
        for x in (clean[2], clean[3]):
            y = [z.clone() if z is x else z for z in clean]
            y[[z is x for z in clean].index(True)][100] = bad
            o, s = L.fs_jagged_attention(*y[:3], off)
            for a, b in zip(L.fs_jagged_attention_backward(*y[:3], o, s, y[3], off), want):
                assert torch.equal(a[:70], b[:70]) and torch.equal(a[370:], b[370:])


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_many_keys_far_below_the_rows_largest(L, d, causal):
    """One key takes nearly all of every row, and thousands of keys of 2^-25 of
    it bring all of the output."""
    n, g = 4000, torch.Generator().manual_seed(d)
    q, k = torch.zeros(n, 1, d), torch.zeros(n, 1, d)
    q[:, 0, 0] = 4.0
    k[1:, 0, 0] = -4.3 - 0.1 * torch.rand(n - 1, generator=g)  # exp(4 k) = 2^-24.8 .. 2^-25.4
    v = 1 + torch.rand(n, 1, d, generator=g)
    v[0] = 0
    q, k, v = (x.to(HF) for x in (q, k, v))
    off = torch.tensor([0, n])
    out, lse = L.fs_jagged_attention(q.cuda(), k.cuda(), v.cuda(), off.cuda(), causal=causal, scale=1.0)
    see = P.sees(n, 0, causal)
    a = (q[:, 0].double() @ k[:, 0].double().T).masked_fill(~see, -math.inf)
    p = torch.softmax(a, 1)
    ref = p @ v[:, 0].double()
    # S is exact but for its product with log2 e (18 2^-24); n terms are summed
    rel = (4 * 18 + 24 + n) * U32
    e = (UT + 2 * rel) * p + see * 2.0 ** -32 * p.amax(1, keepdim=True)
    P.check(out[:, 0], (ref, e @ v[:, 0].double().abs() + UT * ref.abs() + TINY))
    ref = torch.logsumexp(a, 1)
    P.check(lse[0], (ref, rel + 4 * U32 * ref.abs()))
