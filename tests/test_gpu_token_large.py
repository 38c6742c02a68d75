"""A token lookup of more rows than one workgroup each can take in a grid."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_lookup_of_more_workgroups_than_a_grid_has():
    """2^24 + 3 tokens of 4104 columns: 138 GB of output."""
    from jagged_embedding_sparse_amd import lib as L
    n, rows, dim = (1 << 24) + 3, 11, 4104
    if torch.cuda.mem_get_info()[0] < 1.2 * n * dim * 2:
        pytest.skip("the card holds no such output")
    w = torch.arange(rows, device="cuda", dtype=torch.bfloat16)[:, None].expand(rows, dim).contiguous()
    w[:, -1] = 100
    ids = torch.arange(n, device="cuda") % rows
    out = L.fs_token_lookup(w, ids, scale=2.0)
    want = 2 * (torch.arange(n, device="cuda") % rows)
    for col in (0, 2050, dim - 2):
        assert torch.equal(out[:, col].long(), want)
    assert (out[:, -1] == 200).all()
    del out
    torch.cuda.empty_cache()
