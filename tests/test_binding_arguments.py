"""What the binding makes of its arguments, without a GPU (the stubs of
test_binding_streams)."""

import pytest
import torch

from test_binding_streams import calls  # noqa: F401  (a fixture)


def _with_workspace(L):
    """Every call that takes a workspace: its C function, the bytes it needs and
    the call with one given. By name."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    i64 = lambda *x: torch.tensor(x, dtype=torch.int64)  # noqa: E731
    lens, perm, ro, so = i32(1, 2), i32(0, 1), i32(0, 2), i64(0, 1, 3)
    uq = dict(unique=i64(0, 1, 2), unique_offsets=i64(0, 3), seg_offsets=i32(0, 1, 2, 3),
              occ_bm=i32(0, 1, 2), occ_uid=i32(0, 1, 2), counts=i64(3, 0, 3, 0),
              cls=torch.tensor([0, 0, 0], dtype=torch.uint8))
    w = torch.tensor([[1.0] * 16] * 3)
    q = torch.tensor([[[1.0] * 8] * 2] * 3, dtype=torch.bfloat16)
    lse = torch.tensor([[0.0] * 3] * 2)
    bucket = dict(shard_keys=i64(0, 1, 2), shard_bm=i32(0, 1, 2), shard_offsets=i64(0, 3))
    balance = L.balance_workspace_size(2, 1)
    return dict(
        fs_balance_fbs=("_c_balance_fbs", balance, lambda ws: L.fs_balance_fbs(lens, 1, ws=ws)),
        fs_balance_vbs=("_c_balance_vbs", balance, lambda ws: L.fs_balance_vbs(lens, 1, ws=ws)),
        fs_balance_vbs_shares=("_c_balance_shares", balance,
                               lambda ws: L.fs_balance_vbs_shares(lens, 1, i64(1), ws=ws)),
        fs_bucketize_permute=("_c_bucketize", L.bucketize_workspace_size(3, 2, 1, 1),
                              lambda ws: L.fs_bucketize_permute(i64(0, 1, 2)[None], so, [3], perm, ro, 1, ws=ws)),
        fs_unique_collision_split=("_c_unique", L.unique_workspace_size(3, 1, 1),
                                   lambda ws: L.fs_unique_collision_split(
                                       bucket["shard_keys"], bucket["shard_bm"], bucket["shard_offsets"], 3,
                                       [3], 1, ws=ws)),
        fs_collision_split=("_c_collide", L.collision_workspace_size(3, 1, 1),
                            lambda ws: L.fs_collision_split(uq, 3, 1, 1, ws=ws)),
        fs_keyed_transpose=("_c_kt", L.keyed_transpose_workspace_size(1, 2),
                            lambda ws: L.fs_keyed_transpose(i64(1, 2, 3), i32(1, 2)[None], ws=ws)),
        fs_grad_reduce_update=("_c_reduce", L.reduce_workspace_size(3, 16),
                               lambda ws: L.fs_grad_reduce_update([w], [None], 1, [w], 3, uq, "sgd", 0.1, ws=ws)),
        fs_token_sort=("_c_token_sort", L.token_sort_workspace_size(2),
                       lambda ws: L.fs_token_sort(i64(0, 1), 3, ws=ws)),
        fs_token_grad=("_c_token_grad", L.token_grad_workspace_size(3, 16),
                       lambda ws: L.fs_token_grad(uq, w, 3, ws=ws)),
        fs_jagged_attention=("_c_attention", L.attention_workspace_size(3, 2),
                             lambda ws: L.fs_jagged_attention(q, q, q, so, ws=ws)),
        fs_jagged_attention_backward=("_c_attention_bwd", L.attention_backward_workspace_size(3, 2, 2, 2, 8),
                                      lambda ws: L.fs_jagged_attention_backward(q, q, q, q, lse, q, so, ws=ws)))


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int64, torch.float32])
def test_a_workspace_counts_in_bytes(calls, monkeypatch, dtype):  # noqa: F811
    """The C calls get a workspace's bytes whatever its elements are."""
    L, _ = calls
    for name, (fn, need, call) in _with_workspace(L).items():
        got = []
        monkeypatch.setattr(L, fn, lambda *a: got.append(a[-2]) or L.FS_OK)
        size = -(-need // dtype.itemsize)
        call(torch.zeros(size, dtype=dtype))
        assert got == [size * dtype.itemsize] and got[0] >= need, name
        with pytest.raises(AssertionError):
            call(torch.zeros(max(need // dtype.itemsize - 1, 0), dtype=dtype))
        assert len(got) == 1, name


class _On:
    """A tensor of which only the device is asked."""

    def __init__(self, *device):
        self.device = torch.device(*device)

    def get_device(self):
        return -1 if self.device.type == "cpu" else self.device.index


def test_tensors_belong_to_the_current_device(monkeypatch):
    from jagged_embedding_sparse_amd import lib as L
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    here, other, cpu = _On("cuda", 1), _On("cuda", 0), _On("cpu")
    assert L._here(here, None, here) == torch.device("cuda", 1)
    for bad in ((other,), (cpu,), (here, other), (here, None, cpu), (here, here, here, other)):
        with pytest.raises(L.FsError) as e:
            L._here(*bad)
        assert e.value.code == L.FS_ERR_INVALID_ARG


def test_every_tensor_of_a_call_is_checked(calls, monkeypatch):  # noqa: F811
    """Inputs, outputs, flags and workspaces of the token embedding's and the
    attention's calls, all of them given."""
    L, _ = calls
    seen = []
    monkeypatch.setattr(L, "_here", lambda *ts: seen.extend(ts) or torch.device("cpu"))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    i64 = lambda *x: torch.tensor(x, dtype=torch.int64)  # noqa: E731
    w = lambda: torch.ones(3, 16)  # noqa: E731
    h = lambda: torch.ones(3, 2, 8, dtype=torch.bfloat16)  # noqa: E731
    ws = lambda: torch.ones(1 << 16, dtype=torch.uint8)  # noqa: E731
    uq = lambda: dict(unique=i64(0, 1, 2), unique_offsets=i64(0, 3), seg_offsets=i32(0, 1, 2, 3),  # noqa: E731
                      occ_bm=i32(0, 1, 2), occ_uid=i32(0, 1, 2), counts=i64(3, 0, 3, 0))
    side = dict(offsets=i64(0, 1, 3), n_cand=i32(0, 1), valid=torch.ones(3, dtype=torch.uint8))
    sort, grad = uq(), uq()
    del grad["counts"]  # fs_token_grad does not read them
    given = [
        (L.fs_token_lookup, dict(weight=w(), ids=i64(0, 1, 2), out=w(), err=i32(0))),
        (L.fs_token_sort, dict(ids=i64(0, 1, 2), rows=3, out=sort, err=i32(0), ws=ws())),
        (L.fs_token_grad, dict(uq=grad, dout=w(), rows=3, grad=w(), ws=ws())),
        (L.fs_jagged_attention, dict(q=h(), k=h(), v=h(), out=h(), lse=torch.ones(2, 3), err=i32(0),
                                     ws=ws(), **side)),
        (L.fs_jagged_attention_backward, dict(q=h(), k=h(), v=h(), out=h(), lse=torch.ones(2, 3),
                                              dout=h(), dq=h(), dk=h(), dv=h(), err=i32(0), ws=ws(),
                                              **side))]
    for fn, kw in given:
        seen.clear()
        fn(**kw)
        tensors = []
        for x in kw.values():
            tensors += list(x.values()) if isinstance(x, dict) else [x]
        for x in tensors:
            if torch.is_tensor(x):
                assert any(x is y for y in seen), (fn.__name__, [k for k, v in kw.items() if v is x])


FAKE = 1 << 20  # an aligned address that no call below gets to read


def test_grids_of_too_many_threads_are_refused():
    """A grid has fewer than 2^32 threads in one dimension: attention calls of
    more tokens times heads are refused before any launch."""
    import ctypes as C
    from jagged_embedding_sparse_amd import lib as L
    h, n = C.byref(L.FsHeads(FAKE, 0, 0)), 4
    for n_tok, heads, kv, dim, back in ((1 << 28, 8, 8, 8, 0), (1 << 28, 8, 2, 64, 0),
                                        ((1 << 31) - 2, 1, 1, 8, 0), (1 << 26, 32, 8, 128, 0),
                                        (1 << 28, 8, 8, 8, 1), (1 << 27, 8, 8, 128, 1)):
        big = 1 << 62
        if back:
            rc = L._c_attention_bwd(h, h, h, h, FAKE, h, FAKE, n, n_tok, None, None, heads, kv, dim,
                                    L.FS_BF16, 1, 0.1, h, h, h, None, FAKE, big, None)
        else:
            rc = L._c_attention(h, h, h, FAKE, n, n_tok, None, None, heads, kv, dim, L.FS_BF16, 1, 0.1,
                                h, FAKE, None, FAKE, big, None)
        assert rc == L.FS_ERR_UNSUPPORTED, (n_tok, heads, kv, dim, back)


def test_scales_whose_exponents_are_not_finite_are_refused():
    """3e38 is finite, 3e38 log2(e) is not, and 0 times it would be no score."""
    import ctypes as C
    from jagged_embedding_sparse_amd import lib as L
    h, n, n_tok, big = C.byref(L.FsHeads(FAKE, 0, 0)), 4, 50, 1 << 40
    for scale, want in ((3e38, L.FS_ERR_INVALID_ARG), (-2.4e38, L.FS_ERR_INVALID_ARG)):
        assert L._c_attention(h, h, h, FAKE, n, n_tok, None, None, 2, 2, 64, L.FS_BF16, 1, scale, h, FAKE,
                              None, FAKE, big, None) == want
        assert L._c_attention_bwd(h, h, h, h, FAKE, h, FAKE, n, n_tok, None, None, 2, 2, 64, L.FS_BF16, 1,
                                  scale, h, h, h, None, FAKE, big, None) == want
    # nothing launched, nothing refused
    assert L._c_attention(h, h, h, FAKE, n, 0, None, None, 2, 2, 64, L.FS_BF16, 1, 2.3e38, h, FAKE, None,
                          FAKE, big, None) == L.FS_OK
