"""Losses of tokens against a vocabulary's table at their ends: sharp distributions, the
teacher's largest and lowest logits, infinities and NaN, gradients against differences, every
kernel of the large products, many tokens, tables past 32 bits."""

import math

import pytest
import torch

import head_differences as D
import plain_head as H
import plain_ops as P
from test_gpu_token_loss import BF16, F16, F32, KINDS, backward, both, forward, inputs

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


# ---------------------------------------------------------------- infinities and NaN


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n,dim", [(70, 64), (70, 72), (1100, 72)])
@pytest.mark.parametrize("kind", KINDS)
def test_what_a_token_that_takes_part_holds_stays_in_its_loss(kind, n, dim, what):
    x, w, s, dloss = inputs(kind, n, 600, dim, masked=0.3)
    on = ((s["labels"] if kind == "loss" else s["ids"].amax(1)) >= 0)
    clean = forward(x.cuda(), w.cuda(), s)
    bad = int(on.nonzero()[n // 4])
    x[bad, 5] = what
    got = forward(x.cuda(), w.cuda(), s)
    keep = torch.arange(n) != bad
    for k in got:
        assert torch.equal(got[k].cpu()[keep], clean[k].cpu()[keep]), k
    assert not got["loss"][bad].isfinite() and not got["lse"][bad].isfinite()
    dx, _ = backward(x.cuda(), w.cuda(), s, got, dloss)
    assert not dx[bad].isfinite().any() and not dx.cpu()[~on].any()


@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("n,rows", [(70, 600), (1100, 600), (300, 66_000)])
@pytest.mark.parametrize("kind", KINDS)
def test_what_the_table_holds_reaches_tokens_that_take_part(kind, n, rows, what):
    x, w, s, dloss = inputs(kind, n, rows, 64, masked=0.3)
    on = ((s["labels"] if kind == "loss" else s["ids"].amax(1)) >= 0)
    w[rows // 3] = what
    got = forward(x.cuda(), w.cuda(), s)
    dx, _ = backward(x.cuda(), w.cuda(), s, got, dloss)
    for y in (got["loss"], got["lse"]):
        assert not y.cpu()[on].isfinite().any() and not y.cpu()[~on].any()
    assert not dx.cpu()[~on].any()


@pytest.mark.parametrize("n", [40, 300])
@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("kind", KINDS)
def test_losses_gradients_of_either_sign_and_zero(kind, t, n):
    x, w, s, dloss = inputs(kind, n, 500, 72, t)
    dloss *= (torch.arange(n) % 3 - 1).float()
    got, dx, _ = both(x, w, s, dloss)
    assert not dx[1::3].any()


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


# ---------------------------------------------------------------- every kernel


def _held(x, w, s, dloss, dtype=None, scale=1.0):
    """Both directions against the plain forms, computed in 64 bits on the GPU."""
    live = (s["labels"] if "labels" in s else s["ids"].amax(1)) >= 0
    x = x.clone()
    x[~live] = math.nan
    xd, wd = x.cuda(), w.cuda()
    got = forward(xd, wd, s, scale=scale)
    dx, dw = backward(xd, wd, s, got, dloss, dtype=dtype, scale=scale)
    with torch.device("cuda"):
        sd = {k: v.cuda() for k, v in s.items()}
        ref = H.losses(xd, wd, scale, **sd)
        ref.update(H.loss_gradients(xd, wd, got["lse"], dloss.cuda(), dtype or x.dtype, scale, **sd))
        ref = {k: tuple(y.cpu() for y in v) for k, v in ref.items()}
    for name, y in dict(got, dx=dx, dweight=dw).items():
        P.check(y, ref[name], name)


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("dim", [40, 64, 128, 136, 200, 256, 264, 328])
@pytest.mark.parametrize("kind", KINDS)
def test_gradients_of_the_table_in_the_widest_tiles(kind, dim, t):
    """256 tiles of 256 table rows and more: the table's gradient is made in tiles as wide."""
    _held(*inputs(kind, 300, 66_000, dim, t, seed=dim))


@pytest.mark.parametrize("kind,t,dim", [("loss", BF16, 200), ("distill", F16, 264), ("distill", BF16, 128),
                                        ("loss", F16, 100)])
def test_more_pieces_than_one_of_wider_rows(kind, t, dim):
    _held(*inputs(kind, 9000, 70_000, dim, t, masked=0.1, seed=dim))


@pytest.mark.parametrize("n,rows,dim", [(40_001, 300, 72), (300_001, 50, 8)])
@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("kind", KINDS)
def test_many_tokens(kind, t, n, rows, dim):
    """A workgroup packs more tokens than it has threads."""
    _held(*inputs(kind, n, rows, dim, t, top=3, masked=0.4))


@pytest.mark.parametrize("dim", [64, 128, 256, 264])
@pytest.mark.parametrize("top", [1, 9, 64, 65, 200, 256])
def test_many_tokens_entries(top, dim):
    """A wave to a token and its entries, rows of every share of a wave."""
    _held(*inputs("distill", 2100, 400, dim, top=top, seed=top))


@pytest.mark.parametrize("n", [9, 5000])
@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("kind", KINDS)
def test_tables_of_one_and_two_rows(kind, n, rows):
    x, w, s, dloss = inputs(kind, n, rows, 72)
    _held(x, w, s, dloss)
    if rows == 1 and kind == "loss":  # the one row is certain (entries of one id have an entropy)
        got = forward(x.cuda(), w.cuda(), s)
        assert got["loss"].abs().max() <= 4 * P.U32 * (1 + got["lse"].abs().max())


@pytest.mark.parametrize("n", [40, 1100])
@pytest.mark.parametrize("kind", KINDS)
def test_ids_that_32_bits_would_make_good(kind, n):
    x, w, s, dloss = inputs(kind, n, 300, 64, masked=0.0)
    key = "labels" if kind == "loss" else "ids"
    for i, v in enumerate(((1 << 32) + 3, -(1 << 32) + 3, (1 << 63) - 1, -(1 << 63), 1 << 31)):
        s[key][3 * i] = v
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = forward(x.cuda(), w.cuda(), s, err=err)
    assert int(err) != 0
    dx, _ = backward(x.cuda(), w.cuda(), s, got, dloss)
    assert not got["loss"][:15:3].any() and not got["lse"][:15:3].any() and not dx[:15:3].any()
    both(x, w, s, dloss)


@pytest.mark.parametrize("n,rows,dim", [(3, 300, 65536), (3, 300, 65535), (300, 70, 65536)])
@pytest.mark.parametrize("kind", KINDS)
def test_the_widest_rows(kind, n, rows, dim):
    _held(*inputs(kind, n, rows, dim, masked=0.0))


# ---------------------------------------------------------------- past 32 bits


def _in_parts(x, w, s, dloss, step):
    """_held by parts of the tokens, for tokens and a table that are on the GPU."""
    n, t = x.shape[0], x.dtype
    got = forward(x, w, s)
    dx, dw = backward(x, w, s, got, dloss, dtype=F32)
    total, most = 0, 0
    with torch.device("cuda"):
        for lo in range(0, n, step):
            part = {k: v[lo:lo + step] for k, v in s.items()}
            ref = H.losses(x[lo:lo + step], w, **part)
            for name, y in got.items():
                off = (y[lo:lo + step].double() - ref[name][0]).abs()
                assert (off <= ref[name][1]).all(), (name, lo)
            ref = H.loss_gradients(x[lo:lo + step], w, got["lse"][lo:lo + step], dloss[lo:lo + step], t, **part)
            assert ((dx[lo:lo + step].double() - ref["dx"][0]).abs() <= ref["dx"][1]).all(), lo
            total, most = total + ref["dweight"][0], most + ref["dweight"][1]
        assert ((dw.double() - total).abs() <= most).all()


def _on_gpu(kind, n, rows, dim, t=BF16):
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.empty(rows, dim, dtype=t, device="cuda").normal_(0, 2 / math.sqrt(dim), generator=g)
    x = torch.empty(n, dim, dtype=t, device="cuda").normal_(generator=g)
    ids = torch.randint(-rows // 4, rows, (n, 1 if kind == "loss" else 2), generator=g, device="cuda").clamp_min_(-1)
    s = dict(labels=ids[:, 0].contiguous()) if kind == "loss" else \
        dict(ids=ids, teacher=torch.empty(n, 2, device="cuda").normal_(generator=g))
    return x, w, s, torch.rand(n, generator=g, device="cuda") / n


@pytest.mark.parametrize("kind", KINDS)
def test_tokens_past_32_bits(kind):
    """4.5 GB of tokens, and as much of their gradient."""
    _in_parts(*_on_gpu(kind, 1_100_000, 50, 2048), 100_000)


@pytest.mark.parametrize("kind", KINDS)
def test_the_most_tokens(kind):
    x, w, s, dloss = _on_gpu(kind, (1 << 24) - 256, 20, 8)
    _in_parts(x, w, s, dloss, 1 << 21)


@pytest.mark.parametrize("rows,dim,step", [(1_100_000, 2048, 50_000), ((1 << 31) - 1024, 8, 1 << 24)])
@pytest.mark.parametrize("kind", KINDS)
def test_every_row_of_a_table_past_32_bits(kind, rows, dim, step):
    """4.5 and 34 GB of table and as much of its gradient, the second of nearly as many rows as
    a call takes: dx, which reads the table past 32 bits, and every row of the table's gradient."""
    n = 5
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(rows, dim, dtype=BF16, device="cuda")
    for lo in range(0, rows, 1 << 27):
        w[lo:lo + (1 << 27)].normal_(0, 2 / math.sqrt(dim), generator=g)
    x = torch.randn(n, dim, generator=g, device="cuda").to(BF16)
    at = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1])
    s = dict(labels=at) if kind == "loss" else dict(ids=at[:, None].clone(), teacher=torch.zeros(n, 1))
    dloss = torch.full((n,), 0.25)
    dx = torch.full((n, dim), math.nan, dtype=BF16, device="cuda")
    dw = torch.full((rows, dim), math.nan, dtype=BF16, device="cuda")
    got = forward(x, w, s)
    backward(x, w, s, got, dloss, dx=dx, dweight=dw)
    # e's terms of dx are added up within a part of a piece of the table, then by part and piece
    terms = min(rows, 1 << 22) + 1000

    def over_rows(a, b):  # a @ b, whose long sums a product of few rows makes one by one
        return torch.stack([(r[:, None] * b).sum(0) for r in a])

    with torch.device("cuda"):
        live = torch.ones(n, dtype=torch.bool)
        total, size, sums, lse, most = torch.zeros(n, dim, dtype=torch.float64), 0, [], got["lse"], 0
        for lo in range(0, rows, step):
            # the rows' own part of the plain form: labels and entries outside it take part in
            # the tokens' softmax as the given lse, and bring no target
            part, own = w[lo:lo + step], (at >= lo) & (at < lo + step)
            wd = part.double()
            z, e_z = H._scores(x, part, 1.0, live)
            sums.append(torch.logsumexp(z, 1))
            most = torch.maximum(z.abs().amax(1), torch.as_tensor(most))
            p = torch.exp(z - lse.double()[:, None])
            target = torch.zeros_like(p)
            target[own.nonzero()[:, 0].cuda(), (at[own] - lo).cuda()] = 1
            e = 0.25 * (p - target)
            off = 0.25 * (p * (2 * e_z + 6 * P.U32 * (z.abs() + lse.abs()[:, None] + 42) + 4 * P.U32)
                          + (4 + 560) * P.U32 * (p + target))
            e_e = off * (1 + P.u(BF16)) + P.u(BF16) ** 2 * e.abs()  # two numbers of bf16
            have, want = dw[lo:lo + step], e.T @ x.double()
            bound = (e_e.T @ x.double().abs() + 45 * P.U32 * (e.abs().T @ x.double().abs())) * (1 + P.u(BF16))
            bound += P.u(BF16) * want.abs() + P.tiny(BF16)
            assert ((have.double() - want).abs() <= bound).all(), lo
            total += over_rows(e, wd)
            size = size + over_rows(e_e + terms * P.U32 * e.abs(), wd.abs())
        size = size * (1 + P.u(BF16)) + P.u(BF16) * total.abs() + P.tiny(BF16)
        ref = torch.logsumexp(torch.stack(sums), 0)
        z = (x.double() * w[at.cuda()].double()).sum(1)
        e_z = (dim + 4) * P.U32 * float(x.double().abs().sum(1).max()) * float(w[:1 << 20].abs().max())
        # the tiles' sums: 256 scores, and as many tiles as a thread of 64 takes
        e_lse = e_z + 10 * P.U32 * (most + ref.abs()) + (rows / 256 / 64 + 100) * P.U32
    P.check(got["lse"], (ref.cpu(), e_lse.cpu()), "lse")
    P.check(got["loss"], ((ref - z).cpu(), 2 * e_lse.cpu()), "loss")
    P.check(dx, (total.cpu(), size.cpu()), "dx")
