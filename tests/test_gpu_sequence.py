"""The operators together, as a training step uses them: token embedding,
jagged attention and back; and between the sparse step's lookup and update."""

import math

import numpy as np
import pytest
import torch

import plain_ops as P
from harness import host, to_dev
from jagged_embedding_sparse_amd import lib as L
from jagged_embedding_sparse_amd import synth
from jagged_embedding_sparse_amd.step import SparseStep

pytestmark = pytest.mark.gpu


def test_embedding_attention_and_back():
    """Table -> scaled lookup -> attention over the rows' q, k and v parts ->
    its gradients into one projection's gradient -> the table's gradient. Each
    stage is held to the plain form of the inputs it was given."""
    rows, hq, hk, d = 700, 4, 2, 32
    lens, cand = [90, 1, 0, 260, 33], [4, 0, 0, 16, 33]
    g = torch.Generator().manual_seed(5)
    off = torch.tensor([0] + lens).cumsum(0)
    n, width, t = int(off[-1]), (hq + 2 * hk) * d, torch.bfloat16
    table = torch.randn(rows, width, generator=g) / math.sqrt(width)
    ids = (torch.rand(n, generator=g) ** 3 * rows).long()
    ids[::11] = 0  # padding
    ids[5] = rows + 3  # dropped: zeros, and no part in the attention
    scale = math.sqrt(width)

    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dids, doff = ids.cuda(), off.cuda()
    x = L.fs_token_lookup(table.cuda(), dids, scale=scale, dtype=t, err=err)
    assert int(err) == L.FS_EF_ID_RANGE
    ref = P.token_lookup(table, ids, float(np.float32(scale)))
    P.check(x, (ref, ref.abs() * (P.U32 + P.u(t) * (1 + P.U32)) + P.tiny(t)), "lookup")

    valid = ((ids != 0) & (ids < rows)).to(torch.uint8)
    ncand = torch.tensor(cand, dtype=torch.int32)
    qkv = x.view(n, hq + 2 * hk, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    kw = dict(n_cand=ncand.cuda(), valid=valid.cuda(), causal=True)
    out, lse = L.fs_jagged_attention(q, k, v, doff, **kw)
    dout = torch.randn(n, hq, d, generator=g).to(t)
    dx = torch.empty_like(x)
    dqkv = dx.view(n, hq + 2 * hk, d)
    L.fs_jagged_attention_backward(q, k, v, out, lse, dout.cuda(), doff, **kw, dq=dqkv[:, :hq],
                                   dk=dqkv[:, hq:hq + hk], dv=dqkv[:, hq + hk:])
    res = P.attention(*(y.cpu() for y in (q, k, v)), off, ncand, valid, True, d ** -0.5, dout,
                      own_out=True)
    for name, y in dict(out=out, lse=lse, dq=dqkv[:, :hq], dk=dqkv[:, hq:hq + hk],
                        dv=dqkv[:, hq + hk:]).items():
        P.check(y, res[name], name)

    uq = L.fs_token_sort(dids, rows, padding_id=0)
    grad = L.fs_token_grad(uq, dx, rows, scale=scale)
    gref, size = P.token_grad(ids, dx.cpu(), rows, 0, float(np.float32(scale)))
    P.check(grad, (gref, size * (n + 4) * 2.0 ** -53 + gref.abs() * 3 * P.U32 + 1e-40), "table")
    assert (grad[0] == 0).all()


@pytest.mark.parametrize("schedule", ["joined", "serial"])
def test_attention_between_the_steps_lookup_and_update(schedule):
    """The attention reads the step's batch-major rows and offsets as they lie
    on the device, and its gradients drive the step's update."""
    w, seed, heads, d = synth.workload(1), 3, 2, 32
    bt = synth.Batches(w, seed)
    batches = [bt.batch(i) for i in range(2)]
    weight = synth.init_table(w.tables[0].rows, heads * d, "f32", seed, "cuda")
    before = weight.clone()
    cap = max(b["n_tok"] for b in batches)
    step = SparseStep(w, [weight], [None], cap, schedule=schedule)
    dev = [to_dev(b) for b in batches]
    st = step.prologue(dev[0])
    step.join()

    def grads_of(st, b):
        lens = torch.from_numpy(np.diff(b["sample_offsets"]))
        perm = torch.from_numpy(host(st.perm)).long()
        ncand = (lens - torch.from_numpy(b["uih_len"]).long())[perm].int()
        n = b["n_tok"]
        x = (st.out[0][:n] * 100).to(torch.bfloat16).view(n, heads, d)
        off = st.bucket["bal_offsets"]
        out, lse = L.fs_jagged_attention(x, x, x, off, n_cand=ncand.cuda())
        dout = torch.randn(n, heads, d, generator=torch.Generator().manual_seed(1)).to(x.dtype)
        parts = L.fs_jagged_attention_backward(x, x, x, out, lse, dout.cuda(), off,
                                               n_cand=ncand.cuda())
        xc = x.cpu()
        res = P.attention(xc, xc, xc, host(off), ncand, None, True, d ** -0.5, dout, own_out=True)
        for name, y in zip(("out", "dq", "dk", "dv"), (out, *parts)):
            P.check(y, res[name], name)
        grad = torch.zeros(cap, heads * d, device="cuda")
        grad[:n] = sum(y.float() for y in parts).view(n, heads * d)
        return grad

    g0 = grads_of(st, batches[0])
    ids0, perm0 = batches[0]["ids"][0], host(st.perm)
    so = batches[0]["sample_offsets"]
    order = np.concatenate([ids0[so[s]:so[s + 1]] for s in perm0])
    st1 = step.step(dev[1], [g0])
    step.join()
    torch.cuda.synchronize()
    # the rows that the second lookup saw: fp32 SGD, one rounding per operation
    total = torch.zeros(weight.shape, dtype=torch.float64).index_add_(
        0, torch.from_numpy(order), g0[:len(order)].cpu().double())
    want = before.cpu().double() - w.lr * total
    bound = 3 * P.U32 * (before.cpu().double().abs() + w.lr * total.abs())
    P.check(weight, (want, bound), "rows")
    grads_of(st1, batches[1])
    step.epilogue([g0])
    step.join()
    torch.cuda.synchronize()
