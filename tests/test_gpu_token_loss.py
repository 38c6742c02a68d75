"""Losses of tokens against a vocabulary's table, and their gradients, against
the plain 64-bit forms."""

import math

import pytest
import torch

import plain_head as H
import plain_ops as P
from jagged_embedding_sparse_amd import lib as L

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
KINDS = ["loss", "distill"]


def inputs(kind, n, rows, dim, t=BF16, top=5, teacher=F32, seed=0, masked=0.2, pad=-1):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(rows, dim, generator=g) * 2 / math.sqrt(dim)).to(t)
    ids = (torch.rand(n, top if kind == "distill" else 1, generator=g) ** 2 * rows).long()
    x = (torch.randn(n, dim, generator=g)
         + 3 * torch.rand(n, 1, generator=g) * w[ids[:, 0]].float()).to(t)
    off = torch.rand(n, generator=g) < masked
    if kind == "loss":
        s = dict(labels=torch.where(off, pad, ids[:, 0]))
    else:
        gone = torch.rand(ids.shape, generator=g) < 0.2
        s = dict(ids=torch.where(off[:, None] | gone, pad, ids),
                 teacher=(6 * torch.randn(ids.shape, generator=g)).to(teacher))
    return x, w, s, (torch.rand(n, generator=g) + 0.5) / n


def forward(x, w, s, **kw):
    if "labels" in s:
        loss, lse = L.fs_token_loss(x, w, s["labels"].cuda(), **kw)
        return dict(loss=loss, lse=lse)
    loss, lse, logits = L.fs_token_distill(x, w, s["ids"].cuda(), s["teacher"].cuda(), **kw)
    return dict(loss=loss, lse=lse, logits=logits)


def backward(x, w, s, got, dloss, **kw):
    if "labels" in s:
        return L.fs_token_loss_backward(x, w, s["labels"].cuda(), got["lse"], dloss.cuda(), **kw)
    return L.fs_token_distill_backward(x, w, s["ids"].cuda(), s["teacher"].cuda(), got["lse"],
                                       got["logits"], dloss.cuda(), **kw)


def both(x, w, s, dloss, scale=1.0, pad=-1, dtype=None, xd=None, wd=None):
    """Both directions held to the plain forms."""
    xd, wd = x.cuda() if xd is None else xd, w.cuda() if wd is None else wd
    got = forward(xd, wd, s, scale=scale, padding_id=pad)
    ref = H.losses(x, w, scale, pad, **s)
    for name, y in got.items():
        P.check(y, ref[name], name)
    dx, dw = backward(xd, wd, s, got, dloss, scale=scale, padding_id=pad, dtype=dtype)
    ref = H.loss_gradients(x, w, got["lse"].cpu(), dloss, dtype or x.dtype, scale, pad, **s)
    P.check(dx, ref["dx"], "dx")
    P.check(dw, ref["dweight"], "dweight")
    return got, dx, dw


SHAPES = [(1, 1, 8), (1, 5, 1), (2, 300, 3), (3, 7, 64), (17, 300, 64), (63, 256, 64), (64, 255, 128),
          (65, 257, 72), (128, 1000, 136), (129, 511, 100), (200, 513, 40), (257, 2000, 264), (500, 130, 33),
          (31, 3000, 520)]


@pytest.mark.parametrize("n,rows,dim", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [BF16, F16])
def test_every_shape(kind, n, rows, dim, t):
    x, w, s, dloss = inputs(kind, n, rows, dim, t, seed=n)
    both(x, w, s, dloss)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,rows", [(300, 66_000), (200, 132_000)])
def test_wide_tiles(kind, n, rows):
    """Enough tokens and rows for tiles of 256 tokens."""
    x, w, s, dloss = inputs(kind, n, rows, 72, seed=2)
    both(x, w, s, dloss)


def _masked_as_clean(kind, n, rows, dim, t):
    """Both directions held to the plain forms, and the same bits again where the
    masked tokens' rows, lse and dloss are NaN."""
    x, w, s, dloss = inputs(kind, n, rows, dim, t, masked=0.4)
    clean = both(x, w, s, dloss)
    off = (s["labels"] if kind == "loss" else s["ids"].amax(1)) == -1
    x[off], dloss[off] = math.nan, math.nan
    got = forward(x.cuda(), w.cuda(), s)
    for k in got:
        assert torch.equal(got[k], clean[0][k]), k
    got["lse"][off.cuda()] = math.nan
    dx, dw = backward(x.cuda(), w.cuda(), s, got, dloss)
    assert torch.equal(dx, clean[1]) and torch.equal(dw, clean[2])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("n,rows,dim", [(1025, 700, 72), (2500, 300, 264)])
def test_many_tokens_are_packed_together(kind, t, n, rows, dim):
    _masked_as_clean(kind, n, rows, dim, t)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("dim", [64, 100, 128, 200, 320])
def test_wide_tiles_of_every_width(kind, t, dim):
    """256 tokens by 256 rows a tile, some rows of zeros in a tile's end."""
    _masked_as_clean(kind, 1100, 27_000, dim, t)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [500, 27_000])
def test_of_many_tokens_none_takes_part(kind, rows):
    x, w, s, dloss = inputs(kind, 1100, rows, 64, masked=2.0)
    x[:] = math.nan
    got = forward(x.cuda(), w.cuda(), s)
    for y in got.values():
        assert not y.any()
    dx, dw = backward(x.cuda(), w.cuda(), s, got, dloss)
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("kind", KINDS)
def test_one_token_of_many_takes_part(kind):
    x, w, s, dloss = inputs(kind, 1300, 400, 96, masked=0.0)
    key = "labels" if kind == "loss" else "ids"
    keep = s[key][1234].clone()
    s[key][:] = -1
    s[key][1234] = keep
    both(x, w, s, dloss)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [128, 200, 260, 384, 512, 513, 520, 576, 584, 640, 712, 2048])
def test_few_tokens_of_long_rows(kind, dim):
    """Few tiles, of 2 to 32 steps."""
    both(*inputs(kind, 70, 900, dim))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("n,dim", [(1, 64), (63, 128), (65, 64), (300, 192), (1024, 64), (40, 640)])
def test_tokens_read_as_they_lie(kind, n, dim, t):
    """Rows of whole steps, 16-byte aligned, apart; masked ones NaN, ids outside flagged."""
    x, w, s, dloss = inputs(kind, n, 555, dim, t, masked=0.3 if n > 1 else 0.0)
    key = "labels" if kind == "loss" else "ids"
    if n > 4:
        s[key][1] = 555
        s[key][2] = -2
    off = (s[key] if kind == "loss" else s[key].amax(1)) < 0
    off |= (s[key] if kind == "loss" else s[key].amin(1)) >= 555
    buf = torch.full((n, dim + 24), math.nan, dtype=t, device="cuda")
    xd = buf[:, 8:8 + dim]
    xd.copy_(x)
    assert xd.data_ptr() % 16 == 0
    both(x, w, s, dloss, xd=xd)
    want = forward(xd, w.cuda(), s)
    xd[off.cuda()] = math.nan
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = forward(xd, w.cuda(), s, err=err)
    for k in got:
        assert torch.equal(got[k], want[k]), k
        assert not got[k][off.cuda()].any()
    assert int(err) == (L.FS_EF_ID_RANGE if n > 4 else 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [-1.0, 0.0, 0.3, 4.0])
def test_scales(kind, scale):
    x, w, s, dloss = inputs(kind, 90, 700, 64)
    got, dx, dw = both(x, w, s, dloss, scale=scale)
    if scale == 0:
        assert not dx.any() and not dw.any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_types_of_the_tables_gradient(kind, dtype):
    x, w, s, dloss = inputs(kind, 70, 300, 76)
    assert both(x, w, s, dloss, dtype=dtype)[2].dtype == dtype


@pytest.mark.parametrize("teacher", [F32, BF16, F16])
@pytest.mark.parametrize("top", [1, 2, 63, 64, 65, 200, 256])
def test_entries(teacher, top):
    """From one entry to the most, of every type; ids repeat (they are drawn from
    few rows), some entries are missing and some logits -inf."""
    x, w, s, dloss = inputs("distill", 40, 150, 64, F16, top, teacher, seed=top)
    s["teacher"][::3, -1] = -math.inf
    s["teacher"][7] = -math.inf  # a token without any
    got, dx, _ = both(x, w, s, dloss)
    assert got["loss"][7] == 0 and not dx[7].any()


def test_one_entry_is_a_label():
    """A single entry's distribution is 1 at its id."""
    x, w, s, dloss = inputs("loss", 50, 400, 64)
    a, dxa, dwa = both(x, w, s, dloss)
    one = dict(ids=s["labels"][:, None], teacher=torch.full((50, 1), 3.0))
    b, dxb, dwb = both(x, w, one, dloss)
    assert torch.equal(a["lse"], b["lse"]) and (a["loss"] - b["loss"]).abs().max() < 1e-4
    assert torch.equal(dxa, dxb) or (dxa - dxb).abs().max() <= dxa.abs().max() * 2 ** -7


@pytest.mark.parametrize("pad", [-1, 0, 9, 10_000])
@pytest.mark.parametrize("kind", KINDS)
def test_padding_and_ids_outside(kind, pad):
    x, w, s, dloss = inputs(kind, 120, 333, 48, pad=pad, masked=0.3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    both(x, w, s, dloss, pad=pad)
    forward(x.cuda(), w.cuda(), s, padding_id=pad, err=err)
    assert int(err) == 0
    key = "labels" if kind == "loss" else "ids"
    s[key][5] = 333 if pad != 333 else 334
    s[key][6] = -7
    got, dx, _ = both(x, w, s, dloss, pad=pad)
    got = forward(x.cuda(), w.cuda(), s, padding_id=pad, err=err)
    assert int(err) == L.FS_EF_ID_RANGE
    assert not dx[5:7].any() and not got["loss"][5:7].any() and not got["lse"][5:7].any()
    err.zero_()
    backward(x.cuda(), w.cuda(), s, got, dloss, padding_id=pad, err=err)
    assert int(err) == L.FS_EF_ID_RANGE


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 70, 300])
def test_no_token_takes_part(kind, n):
    x, w, s, dloss = inputs(kind, n, 500, 64, masked=2.0)
    x[:] = math.nan
    got = forward(x.cuda(), w.cuda(), s)
    for y in got.values():
        assert not y.any()
    dx, dw = backward(x.cuda(), w.cuda(), s, got, dloss)
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("kind", KINDS)
def test_no_tokens(kind):
    x, w, s, dloss = inputs(kind, 0, 300, 64)
    got = forward(x.cuda(), w.cuda(), s)
    assert got["loss"].shape == got["lse"].shape == (0,)
    dx, dw = backward(x.cuda(), w.cuda(), s, got, dloss)
    assert dx.shape == (0, 64) and dw.shape == (300, 64) and not dw.any()
    dx, none = backward(x.cuda(), w.cuda(), s, got, dloss, dweight=False)
    assert dx.shape == (0, 64) and none is None


@pytest.mark.parametrize("kind", KINDS)
def test_what_masked_tokens_hold_reaches_nobody(kind):
    """Their rows, lse and dloss may be anything, their teachers too."""
    x, w, s, dloss = inputs(kind, 140, 600, 96, masked=0.4)
    clean = both(x, w, s, dloss)
    off = (s["labels"] if kind == "loss" else s["ids"].amax(1)) == -1
    assert off.any()
    x2, d2 = x.clone(), dloss.clone()
    x2[off], d2[off] = math.nan, math.inf
    if kind == "distill":
        s["teacher"][s["ids"] == -1] = math.nan
    got = forward(x2.cuda(), w.cuda(), s)
    for k in got:
        assert torch.equal(got[k], clean[0][k]), k
    got["lse"][off.cuda()] = math.nan
    dx, dw = backward(x2.cuda(), w.cuda(), s, got, d2)
    assert torch.equal(dx, clean[1]) and torch.equal(dw, clean[2])


def test_a_confident_token():
    """A label far above the rest: a loss near 0 and not below it, and a gradient
    of the difference, not of a rounded 1 - 1."""
    x, w, s, dloss = inputs("loss", 64, 300, 64, masked=0.0)
    at = s["labels"]
    x = (4.0 * w[at].float()).to(BF16)
    got, _, _ = both(x, w, s, dloss)
    assert (got["loss"] >= 0).all() and got["loss"].min() < 1e-3


@pytest.mark.parametrize("big", [1e-6, 1.0, 3e4])
@pytest.mark.parametrize("kind", KINDS)
def test_gradients_of_any_size_in_fp16(kind, big):
    """dloss far from 1: e leaves fp16's exponents unless it is scaled."""
    x, w, s, dloss = inputs(kind, 100, 500, 64, F16)
    dloss = dloss * 100 * big
    got = forward(x.cuda(), w.cuda(), s)
    dx, dw = backward(x.cuda(), w.cuda(), s, got, dloss, dtype=F32)
    ref = H.loss_gradients(x, w, got["lse"].cpu(), dloss, F32, **s)
    P.check(dw, ref["dweight"], "dweight")
    if big <= 1:  # dx itself is in fp16
        P.check(dx, ref["dx"], "dx")


def _wider(t, offset, wide):
    n, dim = t.shape
    buf = torch.full((n * wide + offset,), 7.0, dtype=t.dtype, device="cuda")
    view = buf[offset:].view(n, wide)[:, 4:4 + dim]
    view.copy_(t)
    return buf, view


@pytest.mark.parametrize("dim,offset,wide", [(64, 1, 83), (64, 4, 72), (75, 0, 80), (72, 2, 96)])
@pytest.mark.parametrize("kind", KINDS)
def test_rows_anywhere(kind, dim, offset, wide):
    """Rows of wider buffers at any alignment, outputs too; what lies around the
    outputs' rows stays."""
    x, w, s, dloss = inputs(kind, 77, 300, dim)
    _, xd = _wider(x, offset, wide)
    _, wd = _wider(w, offset, wide)
    got, dx, dw = both(x, w, s, dloss, xd=xd, wd=wd)
    for dtype in (BF16, F32):
        b1, dxv = _wider(torch.zeros_like(x), offset, wide)
        b2, dwv = _wider(torch.zeros_like(w, dtype=dtype), offset, wide)
        backward(xd, wd, s, got, dloss, dx=dxv, dweight=dwv)
        assert torch.equal(dxv, dx) and torch.equal(dwv.to(BF16), dw)
        for b, rows in ((b1, 77), (b2, 300)):
            around = torch.ones(rows, wide, dtype=torch.bool)
            around[:, 4:4 + dim] = False
            assert (b[:offset] == 7).all() and (b[offset:].view(rows, wide).cpu()[around] == 7).all()


@pytest.mark.parametrize("kind", KINDS)
def test_one_gradient_alone(kind):
    x, w, s, dloss = inputs(kind, 90, 400, 64)
    got, dx, dw = both(x, w, s, dloss)
    a, none = backward(x.cuda(), w.cuda(), s, got, dloss, dweight=False)
    assert none is None and torch.equal(a, dx)
    none, b = backward(x.cuda(), w.cuda(), s, got, dloss, dx=False)
    assert none is None and torch.equal(b, dw)
    with pytest.raises(L.FsError):
        backward(x.cuda(), w.cuda(), s, got, dloss, dx=False, dweight=False)


@pytest.mark.parametrize("kind", KINDS)
def test_against_differences(kind):
    """The gradients against differences of the calls' own losses: in fp32 steps
    of 2^-4 along a direction that both ends hold exactly in 16 bits."""
    x, w, s, dloss = inputs(kind, 24, 90, 32, F16, masked=0.0)
    g = torch.Generator().manual_seed(3)
    q = lambda t: (t.float() * 64).round().div(64).to(F16)  # noqa: E731
    x, w = q(x.clamp(-4, 4)), q(w.clamp(-4, 4))
    vx = torch.randint(-1, 2, x.shape, generator=g).to(F16) / 64
    vw = torch.randint(-1, 2, w.shape, generator=g).to(F16) / 64
    got = forward(x.cuda(), w.cuda(), s)
    dx, dw = backward(x.cuda(), w.cuda(), s, got, dloss, dtype=F32)

    def total(a, b):
        return (H.losses(a, b, **s)["loss"][0] * dloss.double()).sum()

    for at, direction, grad in (("x", vx, dx), ("w", vw, dw)):
        up = total(x + vx, w) if at == "x" else total(x, w + vw)
        down = total(x - vx, w) if at == "x" else total(x, w - vw)
        want = float(up - down) / 2
        have = float((grad.cpu().double() * direction.double()).sum())
        size = float((grad.cpu().double() * direction.double()).abs().sum())
        # the third derivative's part: steps of 2^-6 in every element move a score
        # by less than 2^-6 * 32 * 4 = 2; measured against the terms' sizes
        assert abs(have - want) <= 0.05 * size, (at, have, want, size)
        # and what the calls say at both ends
        xa, wa = (x + vx, w) if at == "x" else (x, w + vw)
        xb, wb = (x - vx, w) if at == "x" else (x, w - vw)
        own = [(forward(a.cuda(), b.cuda(), s)["loss"].cpu().double() * dloss.double()).sum()
               for a, b in ((xa, wa), (xb, wb))]
        assert abs(float(own[0] - own[1]) / 2 - want) < 1e-4


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,rows", [(100, 700), (400, 66_000)])
def test_equal_calls_give_equal_bits_and_graphs_replay(kind, n, rows):
    x, w, s, dloss = inputs(kind, n, rows, 64)
    xd, wd, dl = x.cuda(), w.cuda(), dloss.cuda()
    sd = {k: v.cuda() for k, v in s.items()}
    want = {k: v.clone() for k, v in forward(xd, wd, sd).items()}
    wantg = [t.clone() for t in backward(xd, wd, sd, want, dl)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = forward(xd, wd, sd)
        grads = backward(xd, wd, sd, got, dl)
    for _ in range(4):
        for t in (*got.values(), *grads):
            t.fill_(3)
        graph.replay()
        eager = backward(xd, wd, sd, want, dl)
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], want[k]), k
        for a, b, c in zip(grads, wantg, eager):
            assert torch.equal(a, b) and torch.equal(b, c)


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(kind):
    sets = [inputs(kind, 200, 900, 64, seed=i) for i in range(2)]
    want = []
    for x, w, s, dloss in sets:
        got = forward(x.cuda(), w.cuda(), s)
        want.append((got, backward(x.cuda(), w.cuda(), s, got, dloss)))
    dev = [(x.cuda(), w.cuda(), {k: v.cuda() for k, v in s.items()}, d.cuda()) for x, w, s, d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    out = []
    for (x, w, s, d), st in zip(dev, streams):
        got = forward(x, w, s, stream=st)
        out.append((got, backward(x, w, s, got, d, stream=st)))
    torch.cuda.synchronize()
    for (a, ga), (b, gb) in zip(want, out):
        for k in a:
            assert torch.equal(a[k], b[k])
        for p, q in zip(ga, gb):
            assert torch.equal(p, q)


@pytest.mark.parametrize("kind", KINDS)
def test_more_pieces_than_one(kind):
    """e of 9000 tokens and 70000 rows is more than one piece of 2^30 bytes; held to
    64-bit products on the GPU, with the sums' bounds."""
    n, rows, dim = 9000, 70_000, 64
    x, w, s, dloss = inputs(kind, n, rows, dim, masked=0.1)
    xd, wd = x.cuda(), w.cuda()
    got = forward(xd, wd, s)
    dx, dw = backward(xd, wd, s, got, dloss, dtype=F32)
    dw_want, dw_size = torch.zeros(rows, dim).cuda().double(), torch.zeros(rows, dim).cuda().double()
    for lo in range(0, n, 1500):
        part = {k: v[lo:lo + 1500] for k, v in s.items()}
        live, target, own = H._targets(rows, **part)
        live, target = live.cuda(), target.cuda()
        a = torch.where(live[:, None], xd[lo:lo + 1500].double(), 0.0)
        z = a @ wd.double().T
        lse = torch.logsumexp(z, 1)
        loss = torch.where(live, own.cuda() - (target * z).sum(1) + lse, 0.0)
        assert (got["loss"][lo:lo + 1500] - loss).abs().max() < 1e-4
        c = torch.where(live, dloss[lo:lo + 1500].cuda().double(), 0.0)[:, None]
        e = c * (torch.exp(z - got["lse"][lo:lo + 1500, None].double()) - target)
        want, size = e @ wd.double(), e.abs() @ wd.double().abs()
        # half a step of e and of the result (bf16 has 8 bits, so a step is 2^-7 of
        # the value at most and half of it 2^-8), and what fp32 sums of many terms
        # of either sign leave
        bound = size * (2.0 ** -8 + 2.0 ** -13) + 2.0 ** -8 * want.abs() + 1e-30
        assert ((dx[lo:lo + 1500].double() - want).abs() <= bound * 1.01).all()
        dw_want += e.T @ a
        dw_size += e.abs().T @ a.abs()
    assert ((dw.double() - dw_want).abs() <= dw_size * (2.0 ** -8 + 2.0 ** -13) + 1e-30).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,dim", [(20, 100), (300, 100)])
def test_a_table_laid_out_in_pieces(kind, n, dim):
    """Rows of 200 bytes are laid out in the workspace, 2^26 bytes of them a time."""
    x, w, s, dloss = inputs(kind, n, 300_000, dim, top=3)
    both(x, w, s, dloss)


@pytest.mark.parametrize("kind", KINDS)
def test_a_capacity_s_workspace_serves_smaller_calls(kind):
    x, w, s, dloss = inputs(kind, 150, 700, 64)
    got, dx, dw = both(x, w, s, dloss)
    ws = torch.empty(L.token_loss_backward_workspace_size(5000, 3000, 64), dtype=torch.uint8,
                     device="cuda").fill_(255)
    again = forward(x.cuda(), w.cuda(), s, ws=ws)
    ws.fill_(255)  # NaN wherever a call reads what it has not written
    dx2, dw2 = backward(x.cuda(), w.cuda(), s, again, dloss, ws=ws)
    assert torch.equal(again["loss"], got["loss"]) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("kind", KINDS)
def test_a_table_past_32_bits(kind):
    """4.5 GB of table and as much of its gradient: first, middle and last rows."""
    rows, dim, n = 1_100_000, 2048, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(rows, dim, dtype=BF16, device="cuda").normal_(0, 2 / math.sqrt(dim), generator=g)
    x = torch.randn(n, dim, generator=g, device="cuda").to(BF16)
    at = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1])
    s = dict(labels=at) if kind == "loss" else dict(ids=at[:, None].clone(), teacher=torch.zeros(n, 1))
    dloss = torch.full((n,), 0.25)
    got = forward(x, w, s)
    z = torch.cat([x.double() @ c.double().T for c in w.split(100_000)], 1).cpu()
    lse = torch.logsumexp(z, 1)
    # the plain forms' bounds: dim fp32 multiply-adds a score, the tiles' sums
    e_z = (dim + 4) * P.U32 * float((x.double().abs() @ w[at].double().abs().T).max()) * 2
    e_lse = e_z + 10 * P.U32 * (z.abs().amax(1) + lse) + (rows / 256 + 100) * P.U32
    P.check(got["lse"], (lse, e_lse), "lse")
    P.check(got["loss"], (lse - z[torch.arange(n), at], 2 * e_lse), "loss")
    dx, dw = backward(x, w, s, got, dloss)
    part = dict(labels=torch.arange(n)) if kind == "loss" else dict(ids=torch.arange(n)[:, None], teacher=s["teacher"])
    ref = H.loss_gradients(x.cpu(), w[at].cpu(), got["lse"].cpu(), dloss, BF16, **part)
    P.check(dw[at], ref["dweight"], "dweight")
    assert dx.isfinite().all()
