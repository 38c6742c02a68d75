"""Layer norm without a GPU: bad arguments are refused on the host, before any
launch, with the documented codes."""

import pytest
import torch

from test_abi_token_attention import FAKE, L, _caller  # noqa: F401  (a fixture)
from test_binding_streams import CURRENT, SIDE, calls  # noqa: F401  (a fixture)


def test_layer_norm_refuses(L):  # noqa: F811
    call = _caller(L._c_layer_norm, "x xt xs n dim weight bias pt eps out ot os mean rstd stream".split(),
                   [FAKE, 0, 0, 10, 64, FAKE, FAKE, 0, 1e-5, FAKE, 1, 0, FAKE, FAKE, None])
    bad, un = L.FS_ERR_INVALID_ARG, L.FS_ERR_UNSUPPORTED
    assert call(n=0) == L.FS_OK and call(n=0, x=None, out=None) == L.FS_OK
    for kw in (dict(x=None), dict(out=None), dict(n=-1), dict(n=(1 << 31) - 1), dict(dim=0), dict(xt=3),
               dict(ot=-1), dict(pt=7), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(xs=252), dict(xs=258), dict(xs=-256), dict(os=126), dict(os=129), dict(x=FAKE + 2),
               dict(out=FAKE + 1), dict(weight=FAKE + 2), dict(bias=FAKE + 1)):
        assert call(**kw) == bad, kw
    assert call(dim=L.FS_MAX_NORM_DIM + 1) == un


def test_layer_norm_backward_refuses(L):  # noqa: F811
    assert L.layer_norm_backward_workspace_size(10, 64) == 0  # few rows need none
    need = L.layer_norm_backward_workspace_size(1000, 64)
    names = "x xt xs n dim mean rstd dout dt ds weight pt dx gs dw db ws ws_bytes stream".split()
    call = _caller(L._c_layer_norm_bwd, names,
                   [FAKE, 0, 0, 1000, 64, FAKE, FAKE, FAKE, 1, 0, FAKE, 0, FAKE, 0, FAKE, FAKE, FAKE, need,
                    None])
    bad, un = L.FS_ERR_INVALID_ARG, L.FS_ERR_UNSUPPORTED
    assert call(n=0, dw=None, db=None) == L.FS_OK
    for kw in (dict(x=None), dict(dout=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(n=-1),
               dict(n=(1 << 31) - 1), dict(dim=0), dict(xt=3), dict(dt=-1), dict(pt=3), dict(xs=252),
               dict(ds=126), dict(gs=254), dict(x=FAKE + 2), dict(dout=FAKE + 1), dict(dx=FAKE + 2),
               dict(weight=FAKE + 2), dict(dw=FAKE + 2), dict(db=FAKE + 1)):
        assert call(**kw) == bad, kw
    assert call(dim=L.FS_MAX_NORM_DIM + 1) == un
    assert call(ws=None) == L.FS_ERR_WORKSPACE and call(ws_bytes=need - 1) == L.FS_ERR_WORKSPACE


def test_workspaces_never_decrease(L):  # noqa: F811
    for dim in (1, 100, 16384):
        sizes = [L.layer_norm_backward_workspace_size(n, dim) for n in range(3000)]
        assert sizes == sorted(sizes) and sizes[-1] > 0
    sizes = [L.layer_norm_backward_workspace_size(500, dim) for dim in range(1, 3000)]
    assert sizes == sorted(sizes)


def _work(L, stream):  # noqa: F811
    kw = dict(stream=stream)
    x, w, m = torch.ones(3, 16), torch.ones(16), torch.ones(3)
    return dict(fs_layer_norm=lambda: L.fs_layer_norm(x, w, w, **kw),
                fs_layer_norm_backward=lambda: L.fs_layer_norm_backward(x, m, m, x, w, **kw))


@pytest.mark.parametrize("name", list(_work(None, None)))
def test_allocations_belong_to_the_stream_of_the_kernels(calls, name):  # noqa: F811
    L, log = calls  # noqa: F811
    _work(L, SIDE)[name]()
    assert log["at"] and set(log["at"]) == {SIDE} and log["kernels"] == [SIDE.cuda_stream]
    assert log["now"] is CURRENT and log["recorded"] == [CURRENT]


def test_every_tensor_is_checked(calls, monkeypatch):  # noqa: F811
    L, _ = calls  # noqa: F811
    seen = []
    monkeypatch.setattr(L, "_here", lambda *ts: seen.extend(ts) or torch.device("cpu"))
    x = lambda: torch.ones(3, 16)  # noqa: E731
    w, m, ws = (lambda: torch.ones(16)), (lambda: torch.ones(3)), torch.ones(1 << 16, dtype=torch.uint8)
    for fn, kw in ((L.fs_layer_norm, dict(x=x(), weight=w(), bias=w(), out=x(), mean=m(), rstd=m())),
                   (L.fs_layer_norm_backward, dict(x=x(), mean=m(), rstd=m(), dout=x(), weight=w(), dx=x(),
                                                   dweight=w(), dbias=w(), ws=ws))):
        seen.clear()
        fn(**kw)
        for k, t in kw.items():
            assert any(t is y for y in seen), (fn.__name__, k)


def test_the_binding_refuses(calls):  # noqa: F811
    """Shapes and types that the C call could not tell."""
    L, log = calls  # noqa: F811
    x, w, m = torch.ones(3, 16), torch.ones(16), torch.ones(3)
    for call in (lambda: L.fs_layer_norm(torch.ones(16), w), lambda: L.fs_layer_norm(x, torch.ones(8)),
                 lambda: L.fs_layer_norm(x, w, w.bfloat16()), lambda: L.fs_layer_norm(x, w, out=torch.ones(2, 16)),
                 lambda: L.fs_layer_norm(x, w, out=x.clone(), dtype=torch.bfloat16),
                 lambda: L.fs_layer_norm(x, w, mean=m.double()),
                 lambda: L.fs_layer_norm_backward(x, m, m, torch.ones(3, 8), w),
                 lambda: L.fs_layer_norm_backward(x, m[:2], m, x, w),
                 lambda: L.fs_layer_norm_backward(x, m, m.double(), x, w),
                 lambda: L.fs_layer_norm_backward(x, m, m, x, w, dx=x.bfloat16()),
                 lambda: L.fs_layer_norm_backward(x, m, m, x, w, dbias=w.half())):
        with pytest.raises(AssertionError):
            call()
    with pytest.raises(L.FsError):
        L.fs_layer_norm(torch.ones(1, 16).expand(3, 16), w)
    with pytest.raises(L.FsError):
        L.fs_layer_norm(x.double(), w)
    assert not log["kernels"]
