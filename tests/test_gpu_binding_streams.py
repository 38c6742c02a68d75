"""The token embedding's and the attention's calls on a stream that is not the
current one, with nothing passed that they can allocate: what they drop goes to
no other stream's work, and the results are those of the current stream."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    from jagged_embedding_sparse_amd import lib
    return lib


def _inputs():
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
    n = 900
    return dict(ids=(torch.rand(n, generator=g) ** 3 * 50).long().cuda(), rows=r(n, 96),
                q=r(n, 4, 64), k=r(n, 2, 64), v=r(n, 2, 64), do=r(n, 4, 64),
                off=torch.tensor([0, 300, 301, 900]).cuda())


def _work(L, x, stream=None):
    uq = L.fs_token_sort(x["ids"], 50, padding_id=0, stream=stream)
    grad = L.fs_token_grad(uq, x["rows"], 50, stream=stream)
    emb = L.fs_token_lookup(grad, x["ids"], scale=2.0, dtype=BF, stream=stream)
    out, lse = L.fs_jagged_attention(x["q"], x["k"], x["v"], x["off"], stream=stream)
    return [grad, emb, out, lse, *L.fs_jagged_attention_backward(
        x["q"], x["k"], x["v"], out, lse, x["do"], x["off"], stream=stream)]


def test_workspaces_of_calls_on_another_stream(L):
    """The other stream is kept behind the current one, which allocates and
    writes blocks of every size that the calls have just dropped."""
    x = _inputs()
    alone = _work(L, x)
    sizes = sorted({L.token_grad_workspace_size(900, 96), L.attention_workspace_size(900, 3),
                    L.attention_backward_workspace_size(900, 3, 4, 2, 64)})
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)  # about a millisecond
        got = _work(L, x, side)
        held = [torch.full((b,), 255, dtype=torch.uint8, device="cuda") for b in sizes for _ in range(8)]
        torch.cuda.synchronize()
        assert all((h == 255).all() for h in held)
        for a, b in zip(alone, got):
            assert torch.equal(a, b)
        del held, got


def test_blocks_stay_with_their_stream(L):
    """The blocks that a call on another stream takes and drops are that
    stream's in the allocator's books."""
    x = _inputs()
    side = torch.cuda.Stream()
    _work(L, x, side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = _work(L, x, side)
    of = {s["address"]: (s["total_size"], s["stream"]) for s in torch.cuda.memory_snapshot()}

    def stream_of(p):
        return next(st for a, (size, st) in of.items() if a <= p < a + size)

    assert {stream_of(t.data_ptr()) for t in got} == {side.cuda_stream}
    assert stream_of(x["q"].data_ptr()) != side.cuda_stream
    torch.cuda.synchronize()
