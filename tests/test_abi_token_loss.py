"""Token losses without a GPU: bad arguments are refused on the host, before any
launch, with the documented codes, and the workspace queries never decrease."""

import pytest
import torch

from test_abi_token_attention import FAKE, L, _caller, _table  # noqa: F401  (a fixture)
from test_binding_streams import CURRENT, SIDE, calls  # noqa: F401  (a fixture)

N, ROWS, DIM = 10, 100, 64


def _tab(L, dtype=1, **kw):  # noqa: F811
    return _table(L, dtype=dtype, **kw)


@pytest.fixture(params=["loss", "loss back", "distill", "distill back"])
def call(L, request):  # noqa: F811
    """(the C call with arguments by name, its workspace's bytes, its outputs)"""
    back = request.param.endswith("back")
    need = (L.token_loss_backward_workspace_size if back else L.token_loss_workspace_size)(N, ROWS, DIM)
    names, ok = "x xs n table".split(), [FAKE, 0, N, _tab(L)]
    if request.param.startswith("loss"):
        names, ok = names + ["labels"], ok + [FAKE]
    else:
        names, ok = names + "ids top teacher tt".split(), ok + [FAKE, 5, FAKE, L.FS_F32]
    if back:
        given = ["lse", "dloss"] if request.param == "loss back" else ["lse", "logits", "dloss"]
        names += given + "scale pad dx dxs dw dwt dws".split()
        ok += [FAKE] * len(given) + [1.0, -1, FAKE, 0, FAKE, L.FS_BF16, 0]
        fn = L._c_token_loss_bwd if request.param == "loss back" else L._c_token_distill_bwd
    else:
        given = ["loss", "lse"] if request.param == "loss" else ["loss", "lse", "logits"]
        names += ["scale", "pad"] + given
        ok += [1.0, -1] + [FAKE] * len(given)
        fn = L._c_token_loss if request.param == "loss" else L._c_token_distill
    names += "err ws ws_bytes stream".split()
    return _caller(fn, names, ok + [None, FAKE, need, None]), need, names, given


def test_refusals(L, call):  # noqa: F811
    call, need, names, given = call
    bad, un = L.FS_ERR_INVALID_ARG, L.FS_ERR_UNSUPPORTED
    wrong = [dict(x=None), dict(x=FAKE + 1), dict(n=-1), dict(n=(1 << 31) - 1), dict(xs=126), dict(xs=129),
             dict(xs=-256), dict(table=None), dict(scale=float("nan")), dict(scale=float("inf")),
             dict(scale=2.4e38), dict(table=_tab(L, rows=0)), dict(table=_tab(L, dim=0)),
             dict(table=_tab(L, weights=None)), dict(table=_tab(L, weights=FAKE + 1)),
             dict(table=_tab(L, stride=126)), dict(table=_tab(L, stride=131))]
    wrong += [{k: None} for k in given]
    wrong += [dict(labels=None)] if "labels" in names else \
        [dict(ids=None), dict(teacher=None), dict(top=0), dict(top=-1), dict(tt=3), dict(tt=-1)]
    if "dx" in names:
        wrong += [dict(dx=None, dw=None), dict(dx=FAKE + 1), dict(dw=FAKE + 1), dict(dxs=126), dict(dxs=131),
                  dict(dwt=3), dict(dwt=-1), dict(dws=126), dict(dws=131),
                  dict(dwt=L.FS_F32, dws=254), dict(dwt=L.FS_F32, dw=FAKE + 2)]
    for kw in wrong:
        assert call(**kw) == bad, kw
    far = [dict(table=_tab(L, dtype=L.FS_F32)), dict(table=_tab(L, dtype=5)),
           dict(table=_tab(L, dim=L.FS_MAX_TOKEN_DIM + 1)), dict(table=_tab(L, rows=(1 << 31) - 1)),
           dict(n=1 << 26), dict(n=1 << 24, table=_tab(L, rows=1 << 20))]
    if "top" in names:
        far.append(dict(top=L.FS_MAX_TOP + 1))
    for kw in far:
        assert call(**kw) == un, kw
    assert call(ws=None) == L.FS_ERR_WORKSPACE and call(ws_bytes=need - 1) == L.FS_ERR_WORKSPACE
    if "dx" not in names:
        assert call(n=0, x=None) == L.FS_OK  # nothing to do


def test_workspaces_never_decrease(L):  # noqa: F811
    lengths = list(range(0, 700)) + [x + d for x in (1024, 4096, 16384, 65536, 1 << 20) for d in range(-2, 3)] \
        + [1 << 22, 1 << 25]
    for f in (L.token_loss_workspace_size, L.token_loss_backward_workspace_size):
        for rows, dim in ((1, 1), (100, 64), (10_007, 200), (131_072, 1024), (1 << 22, 100)):
            sizes = [f(n, rows, dim) for n in lengths]
            assert sizes == sorted(sizes) and sizes[0] > 0, (rows, dim)
        for n, dim in ((1, 8), (129, 72), (5000, 1000)):
            sizes = [f(n, rows, dim) for rows in list(range(1, 3000, 7)) + [1 << 16, 1 << 20, (1 << 31) - 300]]
            assert sizes == sorted(sizes), (n, dim)
    # bounded whatever the vocabulary: e in pieces, sums of cut products
    assert L.token_loss_backward_workspace_size(16384, 1 << 22, 1024) < 7 << 28
    assert L.token_loss_backward_workspace_size(2, 10, 16) < 1 << 17
    # no query overflows
    assert L.token_loss_backward_workspace_size((1 << 31) - 300, (1 << 31) - 300, 65536) > 1 << 40


def _work(L, stream):  # noqa: F811
    kw = dict(stream=stream)
    b16 = torch.bfloat16
    x, w, f = torch.ones(3, 16, dtype=b16), torch.ones(5, 16, dtype=b16), torch.ones(3)
    lab, ids = torch.tensor([0, 1, 2]), torch.tensor([[0, 1], [2, 3], [4, 0]])
    t = torch.ones(3, 2)
    return dict(fs_token_loss=lambda: L.fs_token_loss(x, w, lab, **kw),
                fs_token_loss_backward=lambda: L.fs_token_loss_backward(x, w, lab, f, f, **kw),
                fs_token_distill=lambda: L.fs_token_distill(x, w, ids, t, **kw),
                fs_token_distill_backward=lambda: L.fs_token_distill_backward(x, w, ids, t, f, t, f, **kw))


@pytest.mark.parametrize("name", list(_work(None, None)))
def test_allocations_belong_to_the_stream_of_the_kernels(calls, name):  # noqa: F811
    L, log = calls  # noqa: F811
    _work(L, SIDE)[name]()
    assert log["at"] and set(log["at"]) == {SIDE} and log["kernels"] == [SIDE.cuda_stream]
    assert log["now"] is CURRENT and log["recorded"] == [CURRENT]


def _given():
    b16 = torch.bfloat16
    x = lambda: torch.ones(3, 16, dtype=b16)  # noqa: E731
    w = lambda: torch.ones(5, 16, dtype=b16)  # noqa: E731
    f = lambda: torch.ones(3)  # noqa: E731
    t = lambda: torch.ones(3, 2)  # noqa: E731
    lab, ids = (lambda: torch.tensor([0, 1, 2])), (lambda: torch.tensor([[0, 1], [2, 3], [4, 0]]))
    more = lambda: dict(err=torch.zeros(1, dtype=torch.int32),  # noqa: E731
                        ws=torch.empty(1 << 22, dtype=torch.uint8))
    return dict(
        fs_token_loss=dict(x=x(), weight=w(), labels=lab(), loss=f(), lse=f(), **more()),
        fs_token_loss_backward=dict(x=x(), weight=w(), labels=lab(), lse=f(), dloss=f(), dx=x(), dweight=w(),
                                    **more()),
        fs_token_distill=dict(x=x(), weight=w(), ids=ids(), teacher=t(), loss=f(), lse=f(), logits=t(),
                              **more()),
        fs_token_distill_backward=dict(x=x(), weight=w(), ids=ids(), teacher=t(), lse=f(), logits=t(),
                                       dloss=f(), dx=x(), dweight=w(), **more()))


@pytest.mark.parametrize("name", list(_given()))
def test_every_tensor_is_checked(calls, monkeypatch, name):  # noqa: F811
    L, _ = calls  # noqa: F811
    seen, kw = [], _given()[name]
    monkeypatch.setattr(L, "_here", lambda *ts: seen.extend(ts) or torch.device("cpu"))
    getattr(L, name)(**kw)
    for k, t in kw.items():
        assert any(t is y for y in seen), k


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int64])
@pytest.mark.parametrize("name", list(_given()))
def test_a_workspace_counts_in_bytes(calls, monkeypatch, name, dtype):  # noqa: F811
    L, _ = calls  # noqa: F811
    size = L.token_loss_backward_workspace_size if "backward" in name else L.token_loss_workspace_size
    need, got, kw = size(3, 5, 16), [], _given()[name]
    fn = dict(fs_token_loss="_c_token_loss", fs_token_loss_backward="_c_token_loss_bwd",
              fs_token_distill="_c_token_distill", fs_token_distill_backward="_c_token_distill_bwd")[name]
    monkeypatch.setattr(L, fn, lambda *a: got.append(a[-2]) or L.FS_OK)
    kw["ws"] = torch.zeros(-(-need // dtype.itemsize), dtype=dtype)
    getattr(L, name)(**kw)
    assert got == [kw["ws"].numel() * dtype.itemsize] and got[0] >= need
    kw["ws"] = torch.zeros(need // dtype.itemsize - 1, dtype=dtype)
    with pytest.raises(AssertionError):
        getattr(L, name)(**kw)


def test_the_binding_refuses(calls):  # noqa: F811
    """Shapes and types that the C call could not tell."""
    L, log = calls  # noqa: F811
    bad = {"fs_token_loss": [("x", 0, "t"), ("labels", 0, "int"), ("labels", 0, "short"), ("loss", 0, "double"),
                             ("lse", 0, "short")],
           "fs_token_loss_backward": [("x", 0, "t"), ("lse", 0, "short"), ("dloss", 0, "double"),
                                      ("dx", 0, "short"), ("dweight", 0, "short"), ("labels", 0, "int")],
           "fs_token_distill": [("ids", 0, "int"), ("ids", 0, "short"), ("teacher", 0, "short"),
                                ("logits", 0, "short"), ("logits", 0, "double")],
           "fs_token_distill_backward": [("teacher", 0, "short"), ("logits", 0, "double"), ("lse", 0, "short"),
                                         ("dloss", 0, "short")]}
    make = dict(t=lambda t: t.half(), int=lambda t: t.int(), short=lambda t: t[:-1].contiguous(),
                double=lambda t: t.double())
    for name, changes in bad.items():
        for key, _, how in changes:
            kw = _given()[name]
            kw[key] = make[how](kw[key])
            with pytest.raises(AssertionError):
                getattr(L, name)(**kw)
    kw = _given()["fs_token_loss"]
    kw["x"] = kw["x"][:1].expand(3, 16)
    with pytest.raises(L.FsError):
        L.fs_token_loss(**kw)
    kw = _given()["fs_token_distill"]
    kw["teacher"] = kw["teacher"].double()
    with pytest.raises(L.FsError):
        L.fs_token_distill(**kw)
    assert not log["kernels"]
