"""Plain 64-bit forms of the token embedding and of the jagged attention, on
the CPU, and how far a result rounded to fewer bits may be from them.

Bounds count roundings: one rounding to type t is off by at most half a step,
u(t) = finfo(t).eps / 2 of the value; n fp32 operations on a sum of terms by at
most n 2^-24 of the sum of the terms' sizes."""

import math

import torch

U32 = 2.0 ** -24


def u(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """The spacing of the smallest values, where a relative bound ends: a value
    below the normal range is rounded to a multiple of it, off by at most half."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def token_lookup(w, ids, scale):
    ok = (ids >= 0) & (ids < w.shape[0])
    return torch.where(ok[:, None], w[torch.where(ok, ids, 0)].double() * scale, 0.0)


def token_sort(ids, rows, pad):
    """(unique, seg_offsets, occ_bm, occ_uid) as lists."""
    uq, seg, bm, uid = [], [0], [], []
    by_row = {}
    for i, r in enumerate(ids.tolist()):
        if 0 <= r < rows and r != pad:
            by_row.setdefault(r, []).append(i)
    for r in sorted(by_row):
        bm += by_row[r]
        uid += [len(uq)] * len(by_row[r])
        uq.append(r)
        seg.append(len(bm))
    return uq, seg, bm, uid


def token_grad(ids, dout, rows, pad, scale, base=None):
    """(gradient, sum of the sizes of its terms)"""
    keep = (ids >= 0) & (ids < rows) & (ids != pad)
    g = torch.zeros(rows, dout.shape[1], dtype=torch.float64)
    size = torch.zeros_like(g)
    d = dout[keep].double() * scale
    g.index_add_(0, ids[keep], d)
    size.index_add_(0, ids[keep], d.abs())
    if base is not None:
        g, size = g + base.double(), size + base.double().abs()
    return g, size


def sees(length, cand, causal, valid=None):
    i, j = torch.arange(length)[:, None], torch.arange(length)[None, :]
    s = (j < length - cand) & ((j <= i) | (not causal)) | (i == j)
    if valid is not None:
        s = s & valid[:, None] & valid[None, :]
    return s


def _sample(q, k, v, see, scale):
    """One sample in 64 bits, heads first; see [L, L]."""
    s = (q @ k.transpose(1, 2) * scale).masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, 2)
    p = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    return p, lse


def attention(q, k, v, offsets, cand, valid, causal, scale, dout=None, own_out=False):
    """Per-token results in 64 bits and their bounds for a result in q's type:
    dict of (value, bound) by name. Tokens of no sample hold NaN. own_out: the
    backward pass was given an out within the forward's bound, not the exact
    one rounded."""
    n_tok, hq, d = q.shape
    hk, t = k.shape[1], q.dtype
    group = hq // hk
    nan = math.nan
    ut = u(t)
    names = ["out", "lse"] + (["dq", "dk", "dv"] if dout is not None else [])
    shape = dict(out=(n_tok, hq, d), lse=(hq, n_tok), dq=(n_tok, hq, d), dk=(n_tok, hk, d),
                 dv=(n_tok, hk, d))
    res = {x: (torch.full(shape[x], nan, dtype=torch.float64),
               torch.full(shape[x], nan, dtype=torch.float64)) for x in names}

    def put(name, lo, hi, val, bound):
        for dst, src in zip(res[name], (val, bound)):
            if name == "lse":
                dst[:, lo:hi] = src
            else:
                dst[lo:hi] = src.permute(1, 0, 2)

    for b in range(len(offsets) - 1):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        if hi == lo:
            continue
        ok = torch.ones(hi - lo, dtype=torch.bool) if valid is None else valid[lo:hi] != 0
        see = sees(hi - lo, int(cand[b]) if cand is not None else 0, causal, ok)

        def heads(x, rep=1):  # rows that take no part count as zeros
            x = torch.where(ok[:, None, None], x[lo:hi].double(), 0.0).permute(1, 0, 2)
            return x.repeat_interleave(rep, 0)

        qd, kd, vd = heads(q), heads(k, group), heads(v, group)
        p, lse = _sample(qd, kd, vd, see, scale)
        # relative error of P: of S (d fp32 multiply-adds), of its exponent's
        # argument and of lse (sizes up to S + lse), of exp2 and the sums
        size = abs(scale) * (qd.abs() @ kd.abs().transpose(1, 2))
        top = torch.where(see, size, 0.0).amax((1, 2), keepdim=True)
        rel = ((d + 4) * top + 4 * lse.abs().masked_fill(torch.isinf(lse), 0.0).amax() + 16
               + 4 * math.log2(hi - lo + 1)) * U32 + (hi - lo) * U32
        out = p @ vd
        ov = p @ vd.abs()
        # the forward pass rounds 2^(S - m) with a maximum of 1 over the row, sum at least 1
        low = (see * (tiny(t) / 2)).double() @ vd.abs()
        b_out = (ut + 2 * rel) * ov + low + ut * out.abs() + tiny(t)
        put("out", lo, hi, out, b_out)
        fin = lse.masked_fill(torch.isinf(lse), 0.0).abs()
        put("lse", lo, hi, lse, rel[..., 0] + 4 * U32 * fin)
        if dout is None:
            continue
        do = heads(dout)
        dp = do @ vd.transpose(1, 2)
        dsize = do.abs() @ vd.abs().transpose(1, 2)
        delta = (do * out).sum(2, keepdim=True)
        d_out = (do.abs() * out.abs()).sum(2, keepdim=True)
        off_out = (do.abs() * b_out).sum(2, keepdim=True) if own_out else ut * d_out
        ds = p * (dp - delta)
        # dP and delta in d fp32 steps, out rounded once (the backward's input);
        # P and dS are rounded to t, where they lie below t's normal range (fp16:
        # 2^-14) to a multiple of tiny(t), off by at most half of it each
        under = see * (tiny(t) / 2)
        e_ds = (ut + 2 * rel) * ds.abs() + p * ((d + 4) * U32 * (dsize + d_out) + off_out
                                                + tiny(t) * do.abs().sum(2, keepdim=True)) + under
        e_p = (ut + 2 * rel) * p + under

        def shared(x):
            return x.reshape(hk, group, hi - lo, d).sum(1)

        n_sum = (hi - lo) * group * U32
        dq, s_dq = ds @ kd * scale, ds.abs() @ kd.abs() * abs(scale)
        put("dq", lo, hi, dq, e_ds @ kd.abs() * abs(scale) + n_sum * s_dq + ut * dq.abs() + tiny(t))
        dst = ds.transpose(1, 2)
        dk = shared(dst @ qd * scale)
        put("dk", lo, hi, dk, shared((e_ds.transpose(1, 2) @ qd.abs()
                                      + n_sum * (dst.abs() @ qd.abs())) * abs(scale))
            + ut * dk.abs() + tiny(t))
        dv = shared(p.transpose(1, 2) @ do)
        put("dv", lo, hi, dv, shared(e_p.transpose(1, 2) @ do.abs()
                                     + n_sum * (p.transpose(1, 2) @ do.abs()))
            + ut * dv.abs() + tiny(t))
    return res


def check(got, ref, name=""):
    """got within ref's bound of ref's value, infinities equal."""
    val, bound = ref
    got = got.detach().cpu().double()
    assert got.shape == val.shape, (name, got.shape, val.shape)
    inf = torch.isinf(val)
    assert torch.equal(got[inf], val[inf]), name
    bad = ~((got - val).abs() <= bound) & ~inf
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {at}: got "
                             f"{got[tuple(at)]}, {val[tuple(at)]} +- {bound[tuple(at)]}")
