"""Forks whose rows, pages or shortage are past what one workgroup counts, on the GPU against
their reference."""
import pytest
import torch

import cache_reference as C
from helpers import ensure_built
from modulated_deformable_convolution_amd import cache as K

pytestmark = pytest.mark.gpu
ensure_built()


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


# rows, pages: one workgroup's sizes, and past them in either
@pytest.mark.parametrize("rows,pages", [(3, 4), (2049, 4), (3, 8193)])
@pytest.mark.parametrize("new", [False, True])
def test_tables_without_width(rows, pages, new):
    table = torch.empty(rows, 0, dtype=torch.int32, device="cuda")
    given = torch.full((rows,), 77, dtype=torch.int32, device="cuda")
    t, u, o, m = K.fork_pages(None, table, ints([5] * rows), ints([1] * pages), 16, None,
                              ints([1 + i % 2 * 20 for i in range(rows)]) if new else None, used_out=given)
    assert t.shape == (rows, 0) and u is given and u.tolist() == [0] * rows
    assert o.tolist() == [1] * pages
    assert int(m) == (sum(1 + i % 2 for i in range(rows)) if new else 0)
