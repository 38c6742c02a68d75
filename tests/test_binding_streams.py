"""The binding's calls on a stream that is not the current one: what a call
allocates belongs to the stream its kernels run on, and what it returns is
recorded on the caller's. Without a GPU: allocations and C calls are stubs."""

import inspect

import pytest
import torch


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, torch.device("cuda", 0)


CURRENT, SIDE = Stream(1), Stream(2)


@pytest.fixture
def calls(monkeypatch):
    """The library with CPU memory in the place of the GPU's. Logs which stream
    was current at every allocation and which one every C call was given."""
    from jagged_embedding_sparse_amd import lib as L
    log = dict(now=CURRENT, at=[], kernels=[], recorded=[])

    class under:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.before, log["now"] = log["now"], self.s

        def __exit__(self, *_):
            log["now"] = self.before

    def on_cpu(make):
        def run(*a, device=None, **kw):
            log["at"].append(log["now"])
            return make(*a, **kw)
        return run

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: log["now"])
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, on_cpu(getattr(torch, name)))
    cpu = torch.device("cpu")
    monkeypatch.setattr(L, "_dev", lambda: cpu)
    monkeypatch.setattr(L, "_here", lambda *_: cpu, raising=False)
    monkeypatch.setattr(L, "_stream", lambda s: (s or log["now"]).cuda_stream)
    for name in ("_ptr",):
        monkeypatch.setattr(L, name, lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(L, "_rows_ptr", lambda t: (t.data_ptr(), t.stride(0) * t.element_size()))
    monkeypatch.setattr(L, "_heads_arg", lambda *_: b"")
    monkeypatch.setattr(L, "_used_on", lambda out, s: log["recorded"].append(s), raising=False)
    for name in list(vars(L)):
        if name.startswith("_c_") and not name.endswith("_ws") and name not in ("_c_strerror", "_c_version"):
            monkeypatch.setattr(L, name, lambda *a: log["kernels"].append(a[-1]) or L.FS_OK)
    return L, log


def _work(L, stream):
    """Every call of the binding that allocates, with nothing passed that it can
    allocate itself. By name."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    i64 = lambda *x: torch.tensor(x, dtype=torch.int64)  # noqa: E731
    kw = dict(stream=stream)
    lens, perm, ro, so = i32(1, 2), i32(0, 1), i32(0, 2), i64(0, 1, 3)
    uq = dict(unique=i64(0, 1, 2), unique_offsets=i64(0, 3), seg_offsets=i32(0, 1, 2, 3),
              occ_bm=i32(0, 1, 2), occ_uid=i32(0, 1, 2), counts=i64(3, 0, 3, 0),
              cls=torch.tensor([0, 0, 0], dtype=torch.uint8))
    w = torch.tensor([[1.0] * 16] * 3)
    bucket = dict(shard_keys=i64(0, 1, 2), shard_bm=i32(0, 1, 2), shard_offsets=i64(0, 3))
    q = torch.tensor([[[1.0] * 8] * 2] * 3, dtype=torch.bfloat16)
    lse = torch.tensor([[0.0] * 3] * 2)
    return dict(
        fs_balance_fbs=lambda: L.fs_balance_fbs(lens, 1, **kw),
        fs_balance_vbs=lambda: L.fs_balance_vbs(lens, 1, **kw),
        fs_balance_vbs_shares=lambda: L.fs_balance_vbs_shares(lens, 1, i64(1), **kw),
        fs_rank_cost=lambda: L.fs_rank_cost(lens, perm, ro, **kw),
        fs_bucketize_permute=lambda: L.fs_bucketize_permute(i64(0, 1, 2)[None], so, [3], perm, ro, 1,
                                                            **kw),
        fs_unique_collision_split=lambda: L.fs_unique_collision_split(
            bucket["shard_keys"], bucket["shard_bm"], bucket["shard_offsets"], 3, [3], 1, **kw),
        fs_collision_split=lambda: L.fs_collision_split(
            uq, 3, 1, 1, uq["unique"], uq["unique_offsets"], uq["counts"], 3, **kw),
        fs_jagged_lookup=lambda: L.fs_jagged_lookup([w], 1, uq, 3, **kw),
        fs_ranged_combine=lambda: L.fs_ranged_combine(w, bucket, 1, [16], [torch.float32], [3], 3,
                                                      **kw),
        fs_keyed_transpose=lambda: L.fs_keyed_transpose(i64(1, 2, 3), i32(1, 2)[None], **kw),
        fs_grad_reduce_update=lambda: L.fs_grad_reduce_update([w], [None], 1, [w], 3, uq, "sgd", 0.1,
                                                              **kw),
        fs_token_lookup=lambda: L.fs_token_lookup(w, i64(0, 1), **kw),
        fs_token_sort=lambda: L.fs_token_sort(i64(0, 1), 3, **kw),
        fs_token_grad=lambda: L.fs_token_grad(uq, w, 3, **kw),
        fs_jagged_attention=lambda: L.fs_jagged_attention(q, q, q, so, **kw),
        fs_jagged_attention_backward=lambda: L.fs_jagged_attention_backward(q, q, q, q, lse, q, so,
                                                                            **kw))


NAMES = list(_work(None, None))


def test_every_call_that_allocates_is_listed():
    """A call with a workspace or outputs of its own has no entry here only if
    it allocates neither."""
    from jagged_embedding_sparse_amd import lib as L
    allocates = {n for n, f in vars(L).items() if n.startswith("fs_") and callable(f)
                 and any(x in inspect.getsource(f) for x in ("torch.empty", "torch.zeros", "_ws("))}
    assert allocates == set(NAMES)


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_stream_of_the_kernels(calls, name):
    """A workspace of the current stream's would go to that stream's next
    allocation when the call returns, with the kernels still to run on the
    other stream."""
    L, log = calls
    _work(L, SIDE)[name]()
    assert log["at"] and set(log["at"]) == {SIDE} and log["kernels"] == [SIDE.cuda_stream]
    assert log["now"] is CURRENT and log["recorded"] == [CURRENT]
    log.update(at=[], kernels=[], recorded=[])
    _work(L, None)[name]()
    assert set(log["at"]) == {CURRENT} and log["kernels"] == [CURRENT.cuda_stream]
    assert log["recorded"] == []


def test_results_of_every_shape_are_recorded():
    from jagged_embedding_sparse_amd import lib as L
    seen = []

    class T(torch.Tensor):
        def record_stream(self, s):
            seen.append((int(self[0]), s))

    t = [torch.tensor([i]).as_subclass(T) for i in range(4)]
    for out in (t[0], (t[1], t[2]), [t[3]], dict(a=t[0], b=None), None):
        L._used_on(out, "here")
    assert seen == [(i, "here") for i in (0, 1, 2, 3, 0)]


def test_a_positional_stream_counts(calls):
    L, log = calls
    i32 = torch.tensor([1, 2], dtype=torch.int32)
    L.fs_balance_fbs(i32, 1, None, None, None, None, SIDE)
    assert set(log["at"]) == {SIDE} and log["kernels"] == [SIDE.cuda_stream]
