"""Token embedding on the GPU against the plain 64-bit forms: lookup with
scaling, tokens sorted by row, gradient by the sorted tokens."""

import math

import numpy as np
import pytest
import torch

import plain_ops as P

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def L():
    from jagged_embedding_sparse_amd import lib
    return lib


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _ids(n, rows, seed, skew=2.0, bad=0.0):
    g = _gen(seed)
    ids = (torch.rand(n, generator=g, dtype=torch.float64) ** skew * rows).long().clamp_(0, rows - 1)
    if bad:
        hit = torch.rand(n, generator=g) < bad
        ids[hit] = torch.tensor([-1, rows, -(1 << 62), 1 << 62])[torch.arange(int(hit.sum())) % 4]
    return ids


# ---------------------------------------------------------------- lookup


def _check_lookup(out, w, ids, scale, dtype):
    ref = P.token_lookup(w, ids, float(np.float32(scale)))
    # the fp32 product is rounded, then the output
    bound = ref.abs() * (P.U32 + P.u(dtype) * (1 + P.U32)) + P.tiny(dtype)
    P.check(out, (ref, bound), "lookup")


@pytest.mark.parametrize("ti", TYPES)
@pytest.mark.parametrize("to", TYPES)
@pytest.mark.parametrize("n,rows,dim", [(1, 1, 1), (3, 7, 5), (65, 100, 64), (257, 31, 136),
                                        (1000, 50, 24), (33, 9, 2050)])
def test_lookup(L, ti, to, n, rows, dim):
    w = torch.randn(rows, dim, generator=_gen(dim)).to(ti)
    ids = _ids(n, rows, n, bad=0.1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = L.fs_token_lookup(w.cuda(), ids.cuda(), scale=math.sqrt(dim), dtype=to, err=err)
    assert out.dtype == to
    _check_lookup(out, w, ids, math.sqrt(dim), to)
    off = bool(((ids < 0) | (ids >= rows)).any())
    assert int(err) == (L.FS_EF_ID_RANGE if off else 0)


@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 0), (0, 1), (3, 5), (8, 8), (4, 4)])
@pytest.mark.parametrize("ti,to", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16)])
def test_lookup_strides_and_alignment(L, shift, pad, ti, to):
    n, rows, dim = 130, 40, 72
    wide = torch.randn(rows, shift + dim + pad, generator=_gen(1)).to(ti).cuda()
    w = wide[:, shift:shift + dim]
    buf = torch.full((n, shift + dim + pad), 7.0, dtype=to, device="cuda")
    ids = _ids(n, rows, 3)
    L.fs_token_lookup(w, ids.cuda(), scale=0.5, out=buf[:, shift:shift + dim])
    _check_lookup(buf[:, shift:shift + dim], w.cpu(), ids, 0.5, to)
    assert (buf[:, :shift] == 7).all() and (buf[:, shift + dim:] == 7).all()


def test_lookup_empty_and_rows_past_32_bits(L):
    w = torch.ones(4, 8, device="cuda")
    assert L.fs_token_lookup(w, torch.empty(0, dtype=torch.int64, device="cuda")).shape == (0, 8)
    # rows whose byte offsets pass 2^32: 2^20 + 3 rows of 8 KB
    rows, dim = (1 << 20) + 3, 4096
    big = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([0, rows - 1, (1 << 19) + 1, 1 << 20, rows - 2])
    for i in ids.tolist():
        big[i] = i % 251
    out = L.fs_token_lookup(big, ids.cuda(), scale=1.0)
    assert torch.equal(out.cpu().float(), (ids % 251).float()[:, None].expand(-1, dim))


def test_lookup_carries_infinities_and_nan(L):
    w = torch.tensor([[math.inf, -math.inf, math.nan, 3e38]])
    out = L.fs_token_lookup(w.cuda(), torch.zeros(1, dtype=torch.int64).cuda(), scale=2.0).cpu()[0]
    assert out[0] == math.inf and out[1] == -math.inf and out[2].isnan() and out[3] == math.inf


# ---------------------------------------------------------------- sort


def _sorted_lists(uq):
    U = int(uq["counts"][0])
    assert int(uq["unique_offsets"][0]) == 0 and int(uq["unique_offsets"][1]) == U
    seg = uq["seg_offsets"][:U + 1].tolist()
    return uq["unique"][:U].tolist(), seg, uq["occ_bm"][:seg[-1]].tolist(), \
        uq["occ_uid"][:seg[-1]].tolist()


@pytest.mark.parametrize("n", [0, 1, 2, 63, 64, 65, 1000, 1024, 1025, 4095, 4096, 4097, 16_384,
                               16_385, 20_000, 65_536, 65_537, 70_001, 262_144, 262_145])
@pytest.mark.parametrize("rows,pad", [(1, -1), (1, 0), (300, 0), (50_000, 17), (3_000_000, -1)])
def test_sort(L, n, rows, pad):
    ids = _ids(n, rows, n + rows, skew=3.0, bad=0.05 if n % 2 else 0.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    uq = L.fs_token_sort(ids.cuda(), rows, padding_id=pad, err=err)
    assert _sorted_lists(uq) == P.token_sort(ids, rows, pad)
    assert int(err) == (L.FS_EF_ID_RANGE if ((ids != pad) & ((ids < 0) | (ids >= rows))).any() else 0)


@pytest.mark.parametrize("n", [5, 5000])
def test_sort_nothing_left_and_one_row(L, n):
    ids = torch.full((n,), 9, dtype=torch.int64)
    assert _sorted_lists(L.fs_token_sort(ids.cuda(), 10, padding_id=9)) == ([], [0], [], [])
    assert _sorted_lists(L.fs_token_sort(ids.cuda(), 10)) == \
        ([9], [0, n], list(range(n)), [0] * n)
    assert _sorted_lists(L.fs_token_sort(ids.cuda(), 9)) == ([], [0], [], [])
    # an id outside the table that is the padding id drops without a flag
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.fs_token_sort(ids.cuda(), 9, padding_id=9, err=err)
    assert int(err) == 0


@pytest.mark.parametrize("n", [3000, 9000, 100_000, 300_000])
@pytest.mark.parametrize("rows", [255, 256, 511, 512, 2 ** 18 - 1, 2 ** 18, 2 ** 32 - 2])
def test_sort_at_the_bounds_of_digits(L, n, rows):
    ids = torch.randint(0, rows, (n,), generator=_gen(n))
    ids[::3] = rows - 1 - ids[::3] % 5
    assert _sorted_lists(L.fs_token_sort(ids.cuda(), rows, padding_id=rows - 2)) == \
        P.token_sort(ids, rows, rows - 2)


@pytest.mark.parametrize("n", [4097, 66_000])
def test_sort_drops_whole_tiles(L, n):
    ids = torch.arange(n)
    ids[5:] = -1
    assert _sorted_lists(L.fs_token_sort(ids.cuda(), n)) == \
        ([0, 1, 2, 3, 4], [0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4], [0, 1, 2, 3, 4])
    ids[:] = 7
    assert _sorted_lists(L.fs_token_sort(ids.cuda(), n, padding_id=7)) == ([], [0], [], [])


def test_sort_large_rows(L):
    rows = 2 ** 32 - 2
    ids = torch.tensor([rows - 1, 0, 2 ** 31, rows - 1, rows])
    assert _sorted_lists(L.fs_token_sort(ids.cuda(), rows)) == \
        ([0, 2 ** 31, rows - 1], [0, 1, 2, 4], [1, 2, 0, 3], [0, 1, 2, 2])


# ---------------------------------------------------------------- gradient


def _check_grad(got, ids, dout, rows, pad, scale, base=None):
    t = got.dtype
    ref, size = P.token_grad(ids, dout, rows, pad, float(np.float32(scale)), base)
    # 64-bit sums (n 2^-53 of the terms' sizes), one rounding to fp32, one to the type
    bound = size * (len(ids) + 4) * 2.0 ** -53 + ref.abs() * (P.U32 + P.u(t) * (1 + P.U32)) + P.tiny(t)
    P.check(got, (ref, bound), "grad")


@pytest.mark.parametrize("ti", TYPES)
@pytest.mark.parametrize("to", TYPES)
@pytest.mark.parametrize("n,rows,dim,pad", [(1, 1, 1, -1), (7, 3, 5, 0), (300, 700, 64, 0),
                                            (4097, 90, 40, 3), (5000, 20_000, 136, -1),
                                            (70_000, 2500, 24, 1), (200, 33, 2050, 0),
                                            (9000, 12, 2, -1), (3000, 5, 7, -1), (6000, 30, 9, 2),
                                            (2500, 400, 515, 0), (64, 3, 33, -1), (65, 1, 33, -1)])
def test_grad(L, ti, to, n, rows, dim, pad):
    ids = _ids(n, rows, dim, skew=4.0, bad=0.02)
    dout = torch.randn(n, dim, generator=_gen(n)).to(ti)
    uq = L.fs_token_sort(ids.cuda(), rows, padding_id=pad)
    got = L.fs_token_grad(uq, dout.cuda(), rows, scale=1.7, dtype=to)
    _check_grad(got, ids, dout, rows, pad, 1.7)
    again = L.fs_token_grad(uq, dout.cuda(), rows, scale=1.7, dtype=to)
    assert torch.equal(got, again)


@pytest.mark.parametrize("to", TYPES)
@pytest.mark.parametrize("n,rows,dim", [(0, 5, 8), (50, 9, 16), (9000, 100, 72), (700, 11, 3),
                                        (5000, 40, 13), (300, 20, 517)])
def test_grad_accumulates(L, to, n, rows, dim):
    ids = _ids(n, rows, 5)
    dout = torch.randn(n, dim, generator=_gen(2)).to(torch.bfloat16)
    base = torch.randn(rows, dim, generator=_gen(3)).to(to)
    grad = base.cuda()
    uq = L.fs_token_sort(ids.cuda(), rows, padding_id=0)
    L.fs_token_grad(uq, dout.cuda(), rows, scale=-0.3, grad=grad, accumulate=True)
    _check_grad(grad, ids, dout, rows, 0, -0.3, base)
    untouched = torch.ones(rows, dtype=torch.bool)
    untouched[ids[ids != 0]] = False
    assert torch.equal(grad.cpu()[untouched], base[untouched])


@pytest.mark.parametrize("shift,pad", [(1, 0), (3, 5), (8, 8)])
def test_grad_strides_and_alignment(L, shift, pad):
    n, rows, dim = 500, 60, 72
    ids = _ids(n, rows, 1)
    wide = torch.randn(n, shift + dim + pad, generator=_gen(1)).to(torch.bfloat16).cuda()
    dout = wide[:, shift:shift + dim]
    buf = torch.full((rows, shift + dim + pad), 7.0, device="cuda")
    uq = L.fs_token_sort(ids.cuda(), rows)
    L.fs_token_grad(uq, dout, rows, grad=buf[:, shift:shift + dim])
    _check_grad(buf[:, shift:shift + dim], ids, dout.cpu(), rows, -1, 1.0)
    assert (buf[:, :shift] == 7).all() and (buf[:, shift + dim:] == 7).all()


def test_grad_does_not_read_dropped_tokens(L):
    for n in (40, 6000):
        ids = _ids(n, 50, 4, bad=0.2)
        dout = torch.randn(n, 32, generator=_gen(1))
        drop = (ids == 2) | (ids < 0) | (ids >= 50)
        dout[drop] = math.nan
        uq = L.fs_token_sort(ids.cuda(), 50, padding_id=2)
        got = L.fs_token_grad(uq, dout.cuda(), 50)
        _check_grad(got, ids, dout, 50, 2, 1.0)


def test_grad_one_hot_row_of_many_tokens(L):
    """A row over many chunks: sums of multiples of 2^-10 are exact in 64 bits."""
    n, dim = 100_000, 64
    ids = torch.zeros(n, dtype=torch.int64)
    ids[::7] = 3
    dout = torch.randint(-1000, 1000, (n, dim), generator=_gen(1)).float() / 1024
    got = L.fs_token_grad(L.fs_token_sort(ids.cuda(), 5), dout.cuda(), 5).cpu()
    for r in range(5):
        assert torch.equal(got[r], dout[ids == r].double().sum(0).float())


@pytest.mark.parametrize("length", [63, 64, 65, 128, 129, 200, 513])
def test_grad_rows_at_the_bounds_of_whole_and_shared_sums(L, length):
    """Rows of equal length around the bound of rows summed whole, at every
    offset from a chunk's start; sums of multiples of 2^-10 are exact."""
    for lead in (0, 1, 7, 8, 31):
        n = lead + 9 * length + 5
        ids = torch.cat([torch.arange(lead), lead + torch.arange(n - lead) // length])
        rows = int(ids[-1]) + 2
        dout = torch.randint(-1000, 1000, (n, 40), generator=_gen(lead)).float() / 1024
        got = L.fs_token_grad(L.fs_token_sort(ids.cuda(), rows), dout.cuda(), rows).cpu()
        ref = torch.zeros(rows, 40, dtype=torch.float64).index_add_(0, ids, dout.double())
        assert torch.equal(got, ref.float()), lead


def test_expanded_tensors_and_short_sorts_are_refused(L):
    ids = torch.arange(8, device="cuda")
    one = torch.ones(1, 16, device="cuda")
    for call in (lambda: L.fs_token_lookup(one.expand(8, 16), ids),
                 lambda: L.fs_token_lookup(torch.ones(8, 16, device="cuda"), ids,
                                           out=one.clone().expand(8, 16)),
                 lambda: L.fs_token_grad(L.fs_token_sort(ids, 8), one.expand(8, 16), 8)):
        with pytest.raises(L.FsError):
            call()
    with pytest.raises(AssertionError):
        L.fs_token_grad(L.fs_token_sort(ids[:4], 8), torch.ones(8, 16, device="cuda"), 8)
    with pytest.raises(AssertionError):
        L.fs_token_sort(ids, 8, out=L.fs_token_sort(ids[:4], 8))
    with pytest.raises(L.FsError):
        L.fs_token_lookup(torch.ones(8, 16), ids)
    # a table smaller than the sort's: rows past it are left out
    got = L.fs_token_grad(L.fs_token_sort(ids, 8), torch.ones(8, 16, device="cuda"), 5)
    assert got.shape == (5, 16) and (got == 1).all()


def test_grad_takes_the_dedup_of_a_step(L):
    """The outputs of fs_unique_collision_split for one table and several shards."""
    rows, n, W = 1000, 3000, 8
    ids = _ids(n, rows, 8)
    block = -(-rows // W)
    order = torch.argsort(ids // block, stable=True)
    keys, bm = ids[order].cuda(), order.to(torch.int32).cuda()
    so = torch.searchsorted((ids[order] // block).contiguous(), torch.arange(W + 1)).cuda()
    uq = L.fs_unique_collision_split(keys, bm, so, n, [rows], W)
    dout = torch.randn(n, 128, generator=_gen(9))
    got = L.fs_token_grad(uq, dout.cuda(), rows, W=W)
    _check_grad(got, ids, dout, rows, -1, 1.0)
    assert torch.equal(got, L.fs_token_grad(L.fs_token_sort(ids.cuda(), rows), dout.cuda(), rows))


def test_sorted_tokens_drive_the_frameworks_lookup_and_update(L):
    """fs_token_sort's outputs as a one-table, one-shard batch."""
    rows, n, dim = 500, 2000, 64
    ids = _ids(n, rows, 11)
    w = torch.randn(rows, dim, generator=_gen(1))
    uq = L.fs_token_sort(ids.cuda(), rows)
    out = L.fs_jagged_lookup([w.cuda()], 1, uq, n)[0]
    assert torch.equal(out.cpu(), w[ids])
    dout = torch.randn(n, dim, generator=_gen(2)).cuda()
    wd = w.cuda()
    L.fs_grad_reduce_update([wd], [None], 1, [dout], n, uq, "sgd", 0.5)
    grad = L.fs_token_grad(uq, dout, rows)
    assert torch.equal(wd.cpu(), w - 0.5 * grad.cpu())


def test_a_tied_training_step(L):
    """Lookup, its gradient, and a second use of the table added to it."""
    rows, n, dim = 300, 4500, 48
    ids = _ids(n, rows, 2)
    w = torch.randn(rows, dim, generator=_gen(1)).to(torch.bfloat16).cuda()
    x = L.fs_token_lookup(w, ids.cuda(), scale=math.sqrt(dim), dtype=torch.float32)
    uq = L.fs_token_sort(ids.cuda(), rows, padding_id=0)
    first = L.fs_token_grad(uq, x, rows, scale=math.sqrt(dim))
    both = L.fs_token_grad(uq, x, rows, scale=math.sqrt(dim), grad=first.clone(), accumulate=True)
    _check_grad(first, ids, x.cpu(), rows, 0, math.sqrt(dim))
    _check_grad(both, ids, x.cpu(), rows, 0, math.sqrt(dim), first.cpu())


@pytest.mark.parametrize("n", [200, 5000])
def test_capture_replay_and_streams(L, n):
    """Captured once, replayed on new data, with eager work of the same kind
    between the replays; and two streams at once on workspaces of their own."""
    rows, dim = 400, 96
    w = torch.randn(rows, dim, generator=_gen(1)).to(torch.bfloat16).cuda()
    ids = _ids(n, rows, 1).cuda()
    dout = torch.randn(n, dim, generator=_gen(2)).to(torch.bfloat16).cuda()
    ws1 = torch.empty(L.token_sort_workspace_size(n), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(L.token_grad_workspace_size(n, dim), dtype=torch.uint8, device="cuda")

    def work(ids, dout, out=None, uq=None, grad=None, ws1=None, ws2=None, stream=None):
        o = L.fs_token_lookup(w, ids, scale=3.0, out=out, stream=stream)
        uq = L.fs_token_sort(ids, rows, padding_id=0, out=uq, ws=ws1, stream=stream)
        return o, uq, L.fs_token_grad(uq, dout, rows, grad=grad, ws=ws2, stream=stream)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out, uq, grad = work(ids, dout, ws1=ws1, ws2=ws2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(ids, dout, out, uq, grad, ws1, ws2)
    for r in range(4):
        ids.copy_(_ids(n, rows, 10 + r))
        dout.copy_(torch.randn(n, dim, generator=_gen(20 + r)))
        graph.replay()
        torch.cuda.synchronize()
        o2, _, g2 = work(ids.clone(), dout.clone())
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(grad, g2)
    # the same call on another stream than the current one
    ev = torch.cuda.Event()
    ev.record()
    side.wait_event(ev)
    a = work(ids, dout, ws1=ws1, ws2=ws2, stream=side)
    b = work(ids, dout)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
