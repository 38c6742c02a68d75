"""Jagged attention on the GPU, forward and backward, against the plain
64-bit form."""

import math

import pytest
import torch

import plain_ops as P

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def L():
    from jagged_embedding_sparse_amd import lib
    return lib


class Case:
    def __init__(self, lens, hq, hk, d, t, causal=True, cand=None, masked=0.0, fused=False,
                 behind=0, seed=0, spread=1.0, scale=None):
        g = torch.Generator().manual_seed(seed)
        n = sum(lens) + behind
        off = [0]
        for x in lens:
            off.append(off[-1] + x)
        r = lambda h: (torch.randn(n, h, d, generator=g) * spread).to(t)  # noqa: E731
        if fused:
            qkv = r(hq + 2 * hk)
            self.q, self.k, self.v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            self.q, self.k, self.v = r(hq), r(hk), r(hk)
        self.dout = r(hq)
        self.off, self.n, self.n_real, self.t = torch.tensor(off), n, off[-1], t
        self.cand = None if cand is None else torch.tensor(cand, dtype=torch.int32)
        self.valid = None
        if masked:
            self.valid = (torch.rand(n, generator=g) >= masked).to(torch.uint8)
        self.causal, self.scale = causal, d ** -0.5 if scale is None else scale

    def ref(self, dout=True):
        c = None if self.cand is None else \
            torch.minimum(self.cand.clamp(min=0), (self.off[1:] - self.off[:-1]).int())
        return P.attention(self.q, self.k, self.v, self.off, c, self.valid, self.causal, self.scale,
                           self.dout if dout else None)

    def dev(self):
        def up(x):  # keeps a view a view
            if x is None:
                return None
            if x.is_contiguous():
                return x.cuda()
            base = torch.empty(x.shape[0], x.stride(0), dtype=x.dtype)
            base[:, :] = 0
            d = base.cuda().as_strided(x.shape, x.stride(), x.storage_offset() % x.stride(0))
            return d.copy_(x)
        return dict(q=up(self.q), k=up(self.k), v=up(self.v), offsets=self.off.cuda(),
                    n_cand=up(self.cand), valid=up(self.valid), causal=self.causal,
                    scale=self.scale)

    def run(self, L, backward=True):
        a = self.dev()
        ref = self.ref()
        r = self.n_real
        out, lse = L.fs_jagged_attention(**a)
        got = dict(out=out, lse=lse)
        if backward:
            # out and lse as an exact forward pass would have rounded them
            o = torch.nan_to_num(ref["out"][0]).to(self.t).cuda()
            s = torch.where(ref["lse"][0].isnan(), 0.0, ref["lse"][0]).float().cuda()
            q, k, v = a.pop("q"), a.pop("k"), a.pop("v")
            got["dq"], got["dk"], got["dv"] = L.fs_jagged_attention_backward(
                q, k, v, o, s, self.dout.cuda(), **a)
        for name, x in got.items():
            cut = (lambda y: y[:, :r]) if name == "lse" else (lambda y: y[:r])
            P.check(cut(x), tuple(cut(y) for y in ref[name]), name)
        return got


LENS = [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 0, 300]


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [8, 16, 32, 40, 64, 72, 96, 128])
def test_lengths_and_widths(L, t, causal, d):
    Case(LENS, 2, 2, d, t, causal, seed=d).run(L)


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 2), (6, 1), (3, 3), (8, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_shared_heads(L, hq, hk, causal):
    Case([70, 5, 130], hq, hk, 64, BF, causal, cand=[3, 5, 0], fused=True, seed=hq).run(L)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cand", [[0] * 15, [0, 1, 1, 4, 32, 1, 63, 2, 65, 100, 128, 64, 70, 0, 16],
                                  [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 0, 300]])
def test_candidates(L, causal, cand):
    Case(LENS, 2, 1, 32, HF, causal, cand=cand).run(L)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("masked", [0.02, 0.5, 0.97, 1.1])
def test_tokens_that_take_no_part(L, causal, masked):
    c = Case(LENS, 2, 1, 64, BF, causal, cand=[min(x, 5) for x in LENS], masked=masked, seed=3)
    got = c.run(L)
    dead = c.valid[:c.n_real] == 0
    assert (got["out"][:c.n_real].cpu()[dead] == 0).all()
    assert (got["lse"].cpu()[:, :c.n_real][:, dead] == -math.inf).all()
    for x in ("dq", "dk", "dv"):
        assert (got[x][:c.n_real].cpu()[dead] == 0).all()


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf, "lowest"])
def test_what_masked_tokens_hold_does_not_matter(L, t, poison):
    c = Case([5, 64, 130, 257], 4, 2, 40, t, True, cand=[2, 0, 9, 1], masked=0.3, seed=5)
    clean = c.run(L)
    x = torch.finfo(t).min if poison == "lowest" else poison
    for y in (c.q, c.k, c.v, c.dout):
        y[c.valid == 0] = x
    got = c.run(L)
    for name in clean:
        assert torch.equal(clean[name], got[name]), name


def test_rows_behind_the_last_sample_and_between_none(L):
    c = Case([40, 129], 2, 1, 32, BF, behind=75, seed=1)
    for y in (c.q, c.k, c.v, c.dout):
        y[c.n_real:] = math.nan
    a = c.dev()
    full = lambda *s, dt=BF: torch.full(s, 7.0, dtype=dt, device="cuda")  # noqa: E731
    out, lse = full(c.n, 2, 32), full(2, c.n, dt=torch.float32)
    L.fs_jagged_attention(**a, out=out, lse=lse)
    dq, dk, dv = full(c.n, 2, 32), full(c.n, 1, 32), full(c.n, 1, 32)
    q, k, v = a.pop("q"), a.pop("k"), a.pop("v")
    L.fs_jagged_attention_backward(q, k, v, out, lse, c.dout.cuda(), **a, dq=dq, dk=dk, dv=dv)
    ref, r = c.ref(), c.n_real
    for name, x in dict(out=out, dq=dq, dk=dk, dv=dv).items():
        assert (x[r:] == 7).all(), name
        assert x[:r].isfinite().all(), name
    assert (lse[:, r:] == 7).all()
    P.check(out[:r], tuple(y[:r] for y in ref["out"]))


@pytest.mark.parametrize("spread,scale", [(6.0, 0.25), (1.0, 0.0), (1.0, -0.2), (0.01, 1.0)])
def test_sharp_and_flat_softmax(L, spread, scale):
    """Scores of hundreds (one key takes all), equal scores, a negative scale."""
    Case([3, 64, 200], 2, 2, 64, HF, spread=spread, scale=scale, seed=4).run(L)


def test_infinities_and_nan_in_live_tokens_stay_in_their_sample(L):
    c = Case([33, 70, 64], 2, 2, 32, BF, seed=2)
    c.v[40] = math.nan  # sample 1
    a = c.dev()
    out, _ = L.fs_jagged_attention(**a)
    out = out.cpu()
    assert out[:33].isfinite().all() and out[103:].isfinite().all()
    # a row before it does not see it, but 0 times NaN is NaN in a sum of products (in the
    # plain form too): the contract names only the rows that see it and the other samples
    assert out[40:103].isnan().all()


def test_long_sample(L):
    Case([2100], 1, 1, 64, BF, True, cand=[70], seed=6).run(L)
    Case([1500, 3], 2, 1, 128, HF, False, cand=[70, 1], seed=6).run(L)


def test_split_tiles_with_masks(L):
    """Few key tiles, whose steps are shared by several workgroups."""
    Case([1400], 4, 1, 40, BF, True, cand=[9], masked=0.2, fused=True, seed=2).run(L)
    Case([900, 0, 700], 2, 2, 128, HF, False, cand=[0, 0, 90], masked=0.1, seed=3, behind=70).run(L)


def test_more_tiles_than_the_tables_buckets(L):
    """9000 tokens: 282 tiles of 32 rows; equal keys make every sum easy."""
    n = 9000
    q = torch.zeros(n, 4, 16, dtype=BF, device="cuda")
    v = (torch.arange(n, device="cuda") % 64).to(BF)[:, None, None].expand(n, 1, 16).contiguous()
    out, lse = L.fs_jagged_attention(q, q[:, :1].contiguous(), v, torch.tensor([0, n], device="cuda"))
    mean = torch.cumsum(v[:, 0, 0].double(), 0) / torch.arange(1, n + 1, device="cuda")
    assert ((out[:, :, 0].double() - mean[:, None]).abs() <= 2 * P.u(BF) * mean[:, None]).all()
    ref = torch.arange(1, n + 1, device="cuda").double().log()
    assert ((lse.double() - ref).abs() <= 1e-5).all()


@pytest.mark.parametrize("d", [32, 128])
def test_heads_first_layout(L, d):
    """[heads, n_tok, dim] memory: tokens close together, heads far apart."""
    c = Case([100, 37], 4, 2, d, BF, True, cand=[3, 0], seed=6)
    a = c.dev()
    for x in "qkv":
        a[x] = a[x].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(4, c.n, d, dtype=BF, device="cuda").transpose(0, 1)
    lse = L.fs_jagged_attention(**a, out=out)[1]
    plain, lse2 = L.fs_jagged_attention(**c.dev())
    assert torch.equal(out, plain) and torch.equal(lse, lse2)
    q, k, v = a.pop("q"), a.pop("k"), a.pop("v")
    grads = L.fs_jagged_attention_backward(q, k, v, out, lse, c.dout.cuda(), **a)
    b = c.dev()
    q, k, v = b.pop("q"), b.pop("k"), b.pop("v")
    for x, y in zip(grads, L.fs_jagged_attention_backward(q, k, v, plain, lse, c.dout.cuda(), **b)):
        assert torch.equal(x, y)


def test_expanded_heads_and_other_devices_are_refused(L):
    q = torch.zeros(9, 4, 32, dtype=BF, device="cuda")
    off = torch.tensor([0, 9], device="cuda")
    for k in (q[:, :1].expand(9, 4, 32), q[:1].expand(9, 4, 32)):
        with pytest.raises(L.FsError):
            L.fs_jagged_attention(q, k, q, off)
    with pytest.raises(L.FsError):
        L.fs_jagged_attention(q.cpu(), q, q, off)


def test_two_calls_at_once(L):
    """Forward and backward of two batches on two streams, each with its own
    workspaces, against the same calls one after the other."""
    cases = [Case([300, 20], 4, 2, 64, BF, seed=1), Case([64, 500], 4, 4, 128, HF, False, seed=2)]
    args = [c.dev() for c in cases]
    dos = [c.dout.cuda() for c in cases]

    def work(i, stream=None):
        a = dict(args[i])
        out, lse = L.fs_jagged_attention(**a, stream=stream)
        q, k, v = a.pop("q"), a.pop("k"), a.pop("v")
        return [out, lse, *L.fs_jagged_attention_backward(q, k, v, out, lse, dos[i], **a,
                                                          stream=stream)]
    alone = [work(0), work(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        both = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                both.append(work(i))
        torch.cuda.synchronize()
        for x, y in zip(alone, both):
            assert all(torch.equal(u, w) for u, w in zip(x, y))


def test_many_short_samples(L):
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 9, (2500,), generator=g).tolist()
    Case(lens, 2, 1, 16, BF, True, cand=[min(2, x) for x in lens]).run(L)


def test_gradient_by_differences(L):
    """The kernel's gradient against central differences of the 64-bit loss."""
    c = Case([20, 65], 4, 2, 32, HF, True, cand=[4, 0], masked=0.1, seed=8)
    got = c.run(L)
    base = {x: getattr(c, x).double() for x in "qkv"}

    def loss(kw):
        r = P.attention(kw["q"], kw["k"], kw["v"], c.off, c.cand, c.valid, c.causal, c.scale)
        return (r["out"][0] * c.dout.double()).sum()

    for x in "qkv":
        step = torch.randn(base[x].shape, dtype=torch.float64,
                           generator=torch.Generator().manual_seed(3))
        eps = 1e-4
        slope = (loss({**base, x: base[x] + eps * step})
                 - loss({**base, x: base[x] - eps * step})) / (2 * eps)
        bound = (c.ref()["d" + x][1] * step.abs()).sum() + 1e-5 * (1 + slope.abs())
        assert abs((got["d" + x].cpu().double() * step).sum() - slope) <= bound


def test_equal_calls_give_equal_bits_and_strided_outputs(L):
    c = Case([200, 31, 128], 8, 2, 64, BF, cand=[8, 2, 0], masked=0.05, fused=True, seed=9)
    a = c.dev()
    out, lse = L.fs_jagged_attention(**a)
    out2, lse2 = L.fs_jagged_attention(**a)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    wide = torch.full((c.n, 12, 64), 7.0, dtype=BF, device="cuda")
    o3 = torch.full((c.n, 9, 72), 7.0, dtype=BF, device="cuda")
    L.fs_jagged_attention(**a, out=o3[:, :8, :64])
    assert torch.equal(o3[:, :8, :64], out) and (o3[:, 8:] == 7).all() and (o3[..., 64:] == 7).all()
    q, k, v = a.pop("q"), a.pop("k"), a.pop("v")
    do = c.dout.cuda()
    d1 = L.fs_jagged_attention_backward(q, k, v, out, lse, do, **a)
    L.fs_jagged_attention_backward(q, k, v, out, lse, do, **a, dq=wide[:, :8], dk=wide[:, 8:10],
                                   dv=wide[:, 10:])
    for x, y in zip(d1, (wide[:, :8], wide[:, 8:10], wide[:, 10:])):
        assert torch.equal(x, y)


def test_faulty_offsets_and_counts_are_flagged(L):
    c = Case([20, 30], 1, 1, 32, BF, cand=[25, -1])
    a = c.dev()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = L.fs_jagged_attention(**a, err=err)
    assert int(err) == L.FS_EF_SHAPE  # clamped to [0, length]
    P.check(out, c.ref(False)["out"])
    for off in ([0, 30, 20], [-1, 5, 50], [0, 10, 51], [0, 1 << 40, 50], [40, 0, 50]):
        err.zero_()
        out = torch.full((50, 1, 32), 7.0, dtype=BF, device="cuda")
        a["offsets"] = torch.tensor(off).cuda()
        L.fs_jagged_attention(**a, out=out, err=err)
        assert int(err) == L.FS_EF_SHAPE and (out == 7).all(), off


def test_empty_batches(L):
    e = torch.empty(0, 2, 32, dtype=BF, device="cuda")
    for off in ([0], [0, 0, 0]):
        o = torch.tensor(off, device="cuda")
        out, lse = L.fs_jagged_attention(e, e, e, o)
        assert out.shape == (0, 2, 32) and lse.shape == (2, 0)
        L.fs_jagged_attention_backward(e, e, e, out, lse, e, o)
    q = torch.randn(7, 2, 32, device="cuda").to(BF)
    out = torch.full_like(q, 7)
    L.fs_jagged_attention(q, q, q, torch.tensor([0, 0], device="cuda"), out=out)
    assert (out == 7).all()


def test_capture_replay_and_streams(L):
    """Forward and backward captured together, replayed on new data with eager
    calls between; the same calls on a stream that is not the current one."""
    c = Case([150, 64, 1, 33], 4, 2, 64, BF, cand=[8, 0, 1, 2], seed=1)
    a = c.dev()
    do = c.dout.cuda()
    n = len(c.off) - 1
    ws = torch.empty(L.attention_workspace_size(c.n, n), dtype=torch.uint8, device="cuda")
    wb = torch.empty(L.attention_backward_workspace_size(c.n, n, 4, 2, 64), dtype=torch.uint8,
                     device="cuda")

    def work(a, do, outs=None, ws=None, wb=None, stream=None):
        outs = outs or [None] * 5
        out, lse = L.fs_jagged_attention(**a, out=outs[0], lse=outs[1], ws=ws, stream=stream)
        kw = {x: a[x] for x in ("offsets", "n_cand", "valid", "causal", "scale")}
        d = L.fs_jagged_attention_backward(a["q"], a["k"], a["v"], out, lse, do, **kw, dq=outs[2],
                                           dk=outs[3], dv=outs[4], ws=wb, stream=stream)
        return [out, lse, *d]

    outs = work(a, do, ws=ws, wb=wb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(a, do, outs, ws, wb)
    for r in range(4):
        g = torch.Generator().manual_seed(r)
        for x in (a["q"], a["k"], a["v"], do):
            x.copy_(torch.randn(x.shape, generator=g))
        a["offsets"].copy_(torch.tensor([[0, 1, 100, 200, 248], [0, 0, 248, 248, 248],
                                         [0, 62, 124, 186, 248], [0, 150, 214, 215, 248]][r]))
        graph.replay()
        torch.cuda.synchronize()
        eager = work({k: (v.clone() if torch.is_tensor(v) else v) for k, v in a.items()}, do.clone())
        torch.cuda.synchronize()
        for x, y in zip(outs, eager):
            assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = work(a, do, ws=ws, wb=wb, stream=side)
    e = work(a, do)
    torch.cuda.synchronize()
    for x, y in zip(s, e):
        assert torch.equal(x, y)


def test_offsets_past_32_bits(L):
    """Token and head strides that put rows past 2^31 elements and 2^32 bytes."""
    n, heads, d = 70, 2, 64
    tok = 1 << 25  # elements between tokens: 70 << 26 bytes
    base = torch.empty((n - 1) * tok + 4096, dtype=BF, device="cuda")
    c = Case([n], heads, 1, d, BF, seed=3)
    ref = c.ref()
    q = base.as_strided((n, heads, d), (tok, d, 1))
    k = base.as_strided((n, 1, d), (tok, d, 1), 256)
    v = base.as_strided((n, 1, d), (tok, d, 1), 512)
    do = base.as_strided((n, heads, d), (tok, d, 1), 1024)
    dq = base.as_strided((n, heads, d), (tok, d, 1), 2048)
    for x, y in ((q, c.q), (k, c.k), (v, c.v), (do, c.dout)):
        x.copy_(y)
    out, lse = L.fs_jagged_attention(q, k, v, c.off.cuda())
    P.check(out, ref["out"])
    o, s = ref["out"][0].to(BF).cuda(), ref["lse"][0].float().cuda()
    _, dk, dv = L.fs_jagged_attention_backward(q, k, v, o, s, do, c.off.cuda(), dq=dq)
    for name, x in dict(dq=dq, dk=dk, dv=dv).items():
        P.check(x, ref[name], name)
