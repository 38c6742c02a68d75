"""The operators of a sequence model's training step together: embedding, norm,
attention, norm, loss over the tied table, and back to one gradient of the table;
and a distillation of the same rows."""

import math

import pytest
import torch

import plain_head as H
import plain_ops as P
from jagged_embedding_sparse_amd import lib as L

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def test_a_training_step_with_a_tied_table():
    """Every stage is held to the plain form of the inputs it was given; the
    table's gradient is the loss's with the lookup's added to it."""
    rows, heads, d = 900, 4, 32
    dim, lens = heads * d, [70, 1, 0, 150, 44]
    g = torch.Generator().manual_seed(9)
    off = torch.tensor([0] + lens).cumsum(0)
    n = int(off[-1])
    table = (torch.randn(rows, dim, generator=g) * 2 / math.sqrt(dim)).to(BF16)
    ids = (torch.rand(n, generator=g) ** 3 * rows).long()
    labels = torch.cat([ids[1:], ids[:1]])
    labels[off[1:][off[1:] > 0] - 1] = -1  # a sample's last token predicts nothing
    w1, b1 = 1 + 0.1 * torch.randn(dim, generator=g), 0.1 * torch.randn(dim, generator=g)
    dt, dids, dl, doff = table.cuda(), ids.cuda(), labels.cuda(), off.cuda()

    x = L.fs_token_lookup(dt, dids, scale=4.0, dtype=F32)
    h, mean, rstd = L.fs_layer_norm(x, w1.cuda(), b1.cuda(), dtype=BF16)
    ref = H.norm(x.cpu(), w1, b1, 1e-5, BF16)
    for name, y in zip(("out", "mean", "rstd"), (h, mean, rstd)):
        P.check(y, ref[name], name)
    q = h.view(n, heads, d)
    o, lse_a = L.fs_jagged_attention(q, q, q, doff)
    y = (x + o.view(n, dim).float()).to(BF16)
    z, mean2, rstd2 = L.fs_layer_norm(y, w1.cuda(), b1.cuda())
    loss, lse = L.fs_token_loss(z, dt, dl)
    ref = H.losses(z.cpu(), table, labels=labels)
    P.check(loss, ref["loss"], "loss")
    live = int((labels >= 0).sum())
    dloss = torch.full((n,), 1.0 / live)

    dz, dw = L.fs_token_loss_backward(z, dt, dl, lse, dloss.cuda(), dtype=F32)
    ref = H.loss_gradients(z.cpu(), table, lse.cpu(), dloss, F32, labels=labels)
    P.check(dz, ref["dx"], "dz")
    P.check(dw, ref["dweight"], "dw")
    dy, dg2, db2 = L.fs_layer_norm_backward(y, mean2, rstd2, dz, w1.cuda())
    ref = H.norm_backward(y.cpu(), mean2.cpu(), rstd2.cpu(), dz.cpu(), w1, BF16, F32)
    for name, t in zip(("dx", "dweight", "dbias"), (dy, dg2, db2)):
        P.check(t, ref[name], name)
    parts = L.fs_jagged_attention_backward(q, q, q, o, lse_a, dy.view(n, heads, d), doff)
    dh = sum(t.float() for t in parts).view(n, dim).to(BF16)
    dx, dg1, db1 = L.fs_layer_norm_backward(x, mean, rstd, dh, w1.cuda())
    ref = H.norm_backward(x.cpu(), mean.cpu(), rstd.cpu(), dh.cpu(), w1, F32, F32)
    for name, t in zip(("dx", "dweight", "dbias"), (dx, dg1, db1)):
        P.check(t, ref[name], name)
    dx += dy.float()
    before = dw.cpu().clone()
    uq = L.fs_token_sort(dids, rows)
    L.fs_token_grad(uq, dx, rows, scale=4.0, grad=dw, accumulate=True)
    want, size = P.token_grad(ids, dx.cpu(), rows, -1, 4.0, base=before)
    P.check(dw, (want, size * (n + 4) * 2.0 ** -53 + want.abs() * 3 * P.U32 + 1e-40), "table")
    # a step against the gradient: what the step's own loss says
    assert float(loss.sum()) / live > 0 and torch.isfinite(dw).all()


def test_a_teacher_s_top_logits_drive_a_step():
    """A teacher's forward pass picks the entries that the student is held to."""
    n, rows, dim, top = 180, 700, 96, 24
    g = torch.Generator().manual_seed(4)
    teacher = (torch.randn(rows, dim, generator=g) / 3).to(BF16)
    student = (teacher.float() + 0.05 * torch.randn(rows, dim, generator=g)).to(BF16)
    x = torch.randn(n, dim, generator=g)
    w, b = torch.ones(dim), torch.zeros(dim)
    z, mean, rstd = L.fs_layer_norm(x.cuda(), w.cuda(), b.cuda(), dtype=BF16)
    logits, ids = (z.float() @ teacher.cuda().float().T).topk(top, 1)
    loss, lse, at = L.fs_token_distill(z, student.cuda(), ids, logits, scale=0.5)
    s = dict(ids=ids.cpu(), teacher=logits.cpu())
    ref = H.losses(z.cpu(), student, 0.5, **s)
    for name, y in dict(loss=loss, lse=lse, logits=at).items():
        P.check(y, ref[name], name)
    dloss = torch.full((n,), 4.0 / n)
    dz, dw = L.fs_token_distill_backward(z, student.cuda(), ids, logits, lse, at, dloss.cuda(), scale=0.5)
    ref = H.loss_gradients(z.cpu(), student, lse.cpu(), dloss, BF16, 0.5, **s)
    P.check(dz, ref["dx"], "dz")
    P.check(dw, ref["dweight"], "dw")
    dx, _, _ = L.fs_layer_norm_backward(x.cuda(), mean, rstd, dz, w.cuda())
    P.check(dx, H.norm_backward(x, mean.cpu(), rstd.cpu(), dz.cpu(), w, F32, F32)["dx"], "dx")
