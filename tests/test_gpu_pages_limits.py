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


# ---------------------------------------------------------------- too few pages

MOST = (1 << 31) - 1


def fork_of(rows, pages, width, page, used, new, seed, spread=True):
    """A fork of `rows` rows, some with one parent, whose pages are `pages` of a pool."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).tolist()
    table, counts = [], []
    for b in range(rows):
        n = used(b)
        held = min(-(-n // page), len(order))
        table.append([order.pop() for _ in range(held)] + [-1] * (width - held))
        counts.append(min(n, held * page))
    owners = [0] * pages
    for row in table:
        for p in row:
            if p >= 0:
                owners[p] += 1
    parents = [int(torch.randint(0, rows, (), generator=g)) if spread and i % 3 == 0 else i
               for i in range(rows)]
    return table, counts, owners, page, parents, [new(i) for i in range(rows)]


SHORT = [
    # rows, pages, width, page, tokens of row b, new tokens of row i
    (2100, 2300, 3, 16, lambda b: 5 + b % 12, lambda i: i % 20),           # too few free pages
    (40, 8300, 400, 16, lambda b: 200 * 16 - 3, lambda i: 150 * 16),
    (2100, 9000, 2, 16, lambda b: 3 + b % 28, lambda i: 30),               # too narrow a table
    (40, 9000, 5, 16, lambda b: 3 + b % 70, lambda i: 500 * i),
    (4, 30, 5, 16, lambda b: 20, lambda i: 500),
    (2100, 9000, 2, 16, lambda b: 3, lambda i: MOST if i < 17 else 1),     # more than 31 bits
    (40, 9000, 2, 16, lambda b: 0, lambda i: MOST if i < 32 else 0),       # 2^32 less the table's
    (40, 9000, 0, 16, lambda b: 0, lambda i: MOST if i < 32 else 0),       # 2^32
    (40, 20, 2, 16, lambda b: 0, lambda i: MOST if i < 32 else 0),
    (40, 9000, 7, 1, lambda b: b % 7, lambda i: MOST if i == 6 else 0),    # a row past 31 bits
    (40, 9000, 7, 1, lambda b: b % 7, lambda i: MOST if i % 7 == 6 else 0),
    (40, 300, 7, 1, lambda b: b % 7, lambda i: MOST if i == 6 else 0),
    (40, 9000, 7, 1, lambda b: b % 7, lambda i: MOST - 5 if i == 0 else 0),
]


@pytest.mark.parametrize("case", range(len(SHORT)))
def test_too_few_pages(case):
    """What is missing is counted, at most 2^31 - 1, nothing is copied, and the result is what the
    reference makes of the pages there are."""
    rows, pages, width, page, used, new = SHORT[case]
    table, counts, owners, page, parents, new = fork_of(rows, pages, width, page, used, new, case)
    g = torch.Generator().manual_seed(case)
    pool = torch.randint(0, 256, (2, pages, 32), generator=g, dtype=torch.uint8)
    there = pool.cuda()
    got = K.fork_pages(there, torch.tensor(table, dtype=torch.int32).view(rows, width).cuda(), ints(counts),
                       ints(owners), page, ints(parents), ints(new))
    want = C.fork(pool, table, counts, owners, page, parents, new)
    assert want[3] > 0 and int(got[3]) == min(want[3], MOST)
    for a, b, what in zip(got, want, ("table", "used", "owners")):
        assert a.tolist() == b, what
    assert torch.equal(there.cpu(), pool)
