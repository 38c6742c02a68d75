"""What the norm's and the losses' calls hand back, without a GPU: every output has memory
of its own, so that one may be changed in place while another is kept."""

import inspect

import pytest
import torch

import test_abi_norm
import test_abi_token_loss
from test_binding_streams import NAMES, calls  # noqa: F401  (a fixture)

WORK = [(m, name) for m in (test_abi_norm, test_abi_token_loss) for name in m._work(None, None)]


def _outputs(L, module, name):  # noqa: F811
    """A call's outputs on CPU memory (the C call is a stub)."""
    return [t for t in module._work(L, None)[name]() if t is not None]


@pytest.mark.parametrize("module,name", WORK)
def test_outputs_share_no_memory(calls, module, name):  # noqa: F811
    out = _outputs(calls[0], module, name)
    assert len({t.untyped_storage().data_ptr() for t in out}) == len(out)
    assert all(t._base is None for t in out)


@pytest.mark.parametrize("module,name", WORK)
def test_changing_one_output_leaves_the_others_versions(calls, module, name):  # noqa: F811
    out = _outputs(calls[0], module, name)
    before = [t._version for t in out]
    out[0].zero_()
    assert [t._version for t in out[1:]] == before[1:]


def test_a_loss_may_be_changed_in_place(calls):  # noqa: F811
    """An autograd function around the calls returns one output and saves another."""
    L, _ = calls  # noqa: F811

    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, labels):
            loss, lse = L.fs_token_loss(x, w, labels)
            ctx.save_for_backward(lse)
            return loss

        @staticmethod
        def backward(ctx, dloss):
            lse, = ctx.saved_tensors
            return torch.ones(3, 16, dtype=torch.bfloat16), None, None

    x = torch.ones(3, 16, dtype=torch.bfloat16, requires_grad=True)
    loss = Loss.apply(x, torch.ones(5, 16, dtype=torch.bfloat16), torch.tensor([0, 1, 2]))
    loss.div_(3)
    loss.sum().backward()
    assert (x.grad == 1).all()


def test_every_call_that_allocates_is_tested():
    """Calls that allocate through the binding's helpers are in one of the lists of the tests
    of streams and allocations."""
    from jagged_embedding_sparse_amd import lib as L
    marks = ("torch.empty", "torch.zeros", "_ws(", "_space(", "_out(", "_outs(", "_out_like(")
    allocates = {n for n, f in vars(L).items() if n.startswith("fs_") and callable(f)
                 and any(x in inspect.getsource(f) for x in marks)}
    assert allocates == set(NAMES) | {name for _, name in WORK}
