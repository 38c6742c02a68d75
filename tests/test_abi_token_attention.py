"""Token embedding and jagged attention without a GPU: bad arguments are
refused on the host, before any launch, with the documented codes, and the
workspace queries never decrease."""

import ctypes as C

import pytest

FAKE = 1 << 20  # an aligned address that no call below gets to read


@pytest.fixture(scope="module")
def L():
    from jagged_embedding_sparse_amd import lib
    return lib


def _caller(f, names, ok):
    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[names.index(k)] = v
        return f(*a)
    return call


def _table(L, rows=100, dim=64, dtype=0, stride=0, weights=FAKE):
    t = L.FsTable()
    t.weights, t.rows, t.dim, t.dtype, t.stride = weights, rows, dim, dtype, stride
    return C.byref(t)


def test_token_lookup_refuses(L):
    call = _caller(L._c_token_lookup,
                   "table ids n scale out out_dtype out_stride err stream".split(),
                   [_table(L), FAKE, 10, 1.0, FAKE, L.FS_BF16, 0, None, None])
    bad, un = L.FS_ERR_INVALID_ARG, L.FS_ERR_UNSUPPORTED
    assert call(n=0) == L.FS_OK  # nothing to do, nothing launched
    assert call(n=0, ids=None, out=None) == L.FS_OK
    for kw in (dict(table=None), dict(ids=None), dict(out=None), dict(n=-1), dict(n=(1 << 31) - 1),
               dict(out_dtype=3), dict(out_dtype=-1), dict(out_stride=126), dict(out_stride=129),
               dict(out_stride=-256), dict(out=FAKE + 1), dict(table=_table(L, rows=0)),
               dict(table=_table(L, dim=0)), dict(table=_table(L, dtype=3)),
               dict(table=_table(L, stride=255)), dict(table=_table(L, stride=258)),
               dict(table=_table(L, stride=-4)), dict(table=_table(L, weights=None)),
               dict(table=_table(L, weights=FAKE + 2))):
        assert call(**kw) == bad, kw
    assert call(table=_table(L, dim=L.FS_MAX_TOKEN_DIM + 1)) == un


def test_token_sort_refuses(L):
    need = L.token_sort_workspace_size(10)
    call = _caller(L._c_token_sort,
                   "ids n rows pad unique uo seg bm uid counts err ws ws_bytes stream".split(),
                   [FAKE, 10, 100, -1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, need, None])
    bad = L.FS_ERR_INVALID_ARG
    for kw in (dict(ids=None), dict(n=-1), dict(n=(1 << 31) - 1), dict(rows=0), dict(rows=-5),
               dict(unique=None), dict(uo=None), dict(seg=None), dict(bm=None), dict(uid=None),
               dict(counts=None)):
        assert call(**kw) == bad, kw
    assert call(rows=(1 << 32) - 1) == L.FS_ERR_UNSUPPORTED
    assert call(ws=None) == L.FS_ERR_WORKSPACE
    assert call(ws_bytes=need - 1) == L.FS_ERR_WORKSPACE


def test_token_grad_refuses(L):
    need = L.token_grad_workspace_size(10, 64)
    names = ("unique uo W seg bm uid n dout dd ds scale rows dim grad gd gs acc ws ws_bytes "
             "stream").split()
    call = _caller(L._c_token_grad, names,
                   [FAKE, FAKE, 1, FAKE, FAKE, FAKE, 10, FAKE, 0, 0, 1.0, 100, 64, FAKE, 0, 0, 0,
                    FAKE, need, None])
    bad, un = L.FS_ERR_INVALID_ARG, L.FS_ERR_UNSUPPORTED
    for kw in (dict(unique=None), dict(uo=None), dict(W=0), dict(W=L.FS_MAX_RANKS + 1),
               dict(seg=None), dict(bm=None), dict(uid=None), dict(n=-1), dict(n=(1 << 31) - 1),
               dict(dout=None), dict(dd=3), dict(ds=255), dict(ds=258), dict(rows=0), dict(dim=0),
               dict(grad=None), dict(gd=-1), dict(gs=252), dict(gs=257), dict(grad=FAKE + 2),
               dict(dout=FAKE + 1)):
        assert call(**kw) == bad, kw
    assert call(dim=L.FS_MAX_TOKEN_DIM + 1) == un
    assert call(rows=(1 << 32) - 1) == un
    assert call(ws=None) == L.FS_ERR_WORKSPACE
    assert call(ws_bytes=need - 1) == L.FS_ERR_WORKSPACE


def _heads(L, data=FAKE, tok=0, head=0):
    return C.byref(L.FsHeads(data, tok, head))


NAMES = ("q k v offsets n n_tok n_cand valid heads kv_heads dim dtype causal scale out lse err ws "
         "ws_bytes stream").split()
NAMES_BWD = ("q k v out lse dout offsets n n_tok n_cand valid heads kv_heads dim dtype causal "
             "scale dq dk dv err ws ws_bytes stream").split()


@pytest.fixture(params=["forward", "backward"])
def attention(L, request):
    h = _heads(L)
    if request.param == "forward":
        need = L.attention_workspace_size(50, 4)
        ok = [h, h, h, FAKE, 4, 50, None, None, 8, 2, 64, L.FS_BF16, 1, 0.1, h, FAKE, None, FAKE,
              need, None]
        return _caller(L._c_attention, NAMES, ok), ["q", "k", "v", "out"], need
    need = L.attention_backward_workspace_size(50, 4, 8, 2, 64)
    ok = [h, h, h, h, FAKE, h, FAKE, 4, 50, None, None, 8, 2, 64, L.FS_BF16, 1, 0.1, h, h, h, None,
          FAKE, need, None]
    return _caller(L._c_attention_bwd, NAMES_BWD, ok), \
        ["q", "k", "v", "out", "dout", "dq", "dk", "dv"], need


def test_attention_refuses(L, attention):
    call, arrays, need = attention
    bad, un = L.FS_ERR_INVALID_ARG, L.FS_ERR_UNSUPPORTED
    for kw in (dict(offsets=None), dict(n=-1), dict(n=L.FS_MAX_SAMPLES + 1), dict(n_tok=-1),
               dict(n_tok=(1 << 31) - 1), dict(heads=0), dict(kv_heads=0), dict(kv_heads=3),
               dict(kv_heads=16), dict(lse=None), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert call(**kw) == bad, kw
    for kw in (dict(dtype=L.FS_F32), dict(dtype=7), dict(dim=0), dict(dim=4), dict(dim=60),
               dict(dim=136), dict(heads=2 * L.FS_MAX_HEADS)):
        assert call(**kw) == un, kw
    for x in arrays:
        for h in (None, _heads(L, None), _heads(L, FAKE + 8), _heads(L, tok=1032),
                  _heads(L, head=136), _heads(L, tok=112), _heads(L, head=112),
                  _heads(L, tok=-1024)):
            assert call(**{x: h}) == bad, x
    assert call(ws=None) == L.FS_ERR_WORKSPACE
    assert call(ws_bytes=need - 1) == L.FS_ERR_WORKSPACE
    assert call(n=0) == L.FS_OK and call(n_tok=0) == L.FS_OK  # nothing launched


def test_workspace_queries_never_decrease(L):
    prev = [0] * 4
    for n in list(range(0, 300)) + [4095, 4096, 4097, 5000, 65_535, 65_536, 65_537, 70_000, 1 << 20]:
        now = [L.token_sort_workspace_size(n), L.token_grad_workspace_size(n, 100),
               L.attention_workspace_size(n, 16), L.attention_backward_workspace_size(n, 16, 4, 2, 64)]
        assert all(a >= b for a, b in zip(now, prev)), n
        prev = now
    for dim in range(1, 1100):
        assert L.token_grad_workspace_size(1000, dim) <= L.token_grad_workspace_size(1000, dim + 1)
    assert L.attention_workspace_size(100, 5) <= L.attention_workspace_size(100, 6)
    assert L.attention_backward_workspace_size(100, 5, 2, 2, 64) <= \
        L.attention_backward_workspace_size(100, 5, 4, 2, 64)
    for kv in (1, 3, 8):  # the parts of long tiles: fewer as the batch grows
        prev = 0
        for n in list(range(0, 70_000, 97)) + [1 << 17, 1 << 20]:
            now = L.attention_backward_workspace_size(n, 4, 8, kv, 128)
            assert now >= prev, (kv, n)
            prev = now
