"""The 4-bit cache's reference against what the definition says."""
import math

import pytest
import torch

import cache_reference as C

GRID = sorted({s * m for m in C.MAGNITUDES for s in (-1, 1)})


def test_codes_are_nearest_and_ties_go_to_even_codes():
    x = torch.linspace(-7, 7, 2801, dtype=torch.float64)          # steps of 0.005: ties among them
    code = C.block_codes(x[:, None], torch.zeros(2801, 1, dtype=torch.int64))[:, 0]
    for v, c in zip(x.tolist(), code.tolist()):
        got = C.MAGNITUDES[c & 7] * (-1 if c & 8 else 1)
        best = min(abs(min(max(v, -6), 6) - g) for g in GRID)
        assert abs(abs(min(max(v, -6), 6) - got) - best) < 1e-12
    for tie, want in ((0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)):
        t = torch.tensor([[tie], [-tie]], dtype=torch.float64)
        assert C.block_codes(t, torch.zeros(2, 1, dtype=torch.int64))[:, 0].tolist() == [want, want + 8]


@pytest.mark.parametrize("dtype", list(C.LIMITS), ids=str)
def test_exponents_are_the_smallest(dtype):
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(500, 72, generator=g) * torch.exp(4 * torch.randn(500, 1, generator=g))).to(dtype)
    x = torch.where(x.isfinite(), x, torch.ones_like(x))
    e = C.block_exponents(x, dtype)
    lo, hi = C.LIMITS[dtype]
    for c in range(3):
        top = x[:, 32 * c:32 * c + 32].double().abs().amax(-1)
        v = e[:, c].double()
        assert ((top <= 7 * 2 ** v) | (v == hi)).all()
        assert ((top > 7 * 2 ** (v - 1)) | (v == lo)).all()


def test_nothing_is_off_by_more_than_half_a_step():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(400, 64, generator=g)
    r = C.rounded(x, torch.float32)
    e = torch.repeat_interleave(2.0 ** C.block_exponents(x, torch.float32).double(), 32, -1)
    y = x.double().abs() / e
    half = torch.where(y < 2, 0.25, torch.where(y < 4, 0.5, 1.0))
    assert ((r - x.double()).abs() / e <= half).all()


@pytest.mark.parametrize("dim,page", [(8, 16), (40, 16), (64, 32), (72, 16), (96, 16), (128, 64)])
def test_layout_is_a_permutation(dim, page):
    heads, n = 2, -(-dim // 32)
    seen = {}
    for h in range(heads):
        for t in range(page):
            for c in range(32 * n):
                k, v, ke, ve, s = C.value_places(dim, page, h, t, c)
                for at, what in ((k, "k"), (v, "v")):
                    assert seen.setdefault((at, s), (what, h, t, c)) == (what, h, t, c)
                for at, what in ((ke, "ke"), (ve, "ve")):
                    assert seen.setdefault((at, -1), (what, h, t, c // 32)) == (what, h, t, c // 32)
    assert max(at for at, _ in seen) < C.page_bytes(heads, dim, page)
    spare = C.page_bytes(heads, dim, page) - len({at for at, _ in seen})
    assert spare == (heads * page if n == 3 else 0)


def test_written_tokens_are_read_back():
    g = torch.Generator().manual_seed(2)
    heads, dim, page = 2, 40, 16
    pool = torch.randint(0, 256, (3, C.page_bytes(heads, dim, page)), generator=g, dtype=torch.uint8)
    k, v = (torch.randn(5, heads, dim, generator=g) for _ in range(2))
    k[3, 1, 7] = math.nan
    table = torch.tensor([[2, -1], [0, 1]])
    C.store(pool, heads, dim, page, k, v, table, [3, 18], [0, 3, 5], torch.float32)
    rk, rv = C.rounded_pair(k, v, torch.float32)
    for b, places, rows in ((0, [0, 1, 2], slice(0, 3)), (1, [16, 17], slice(3, 5))):
        a, c, there = C.tokens(pool, heads, dim, page, table, b, places)
        assert there.all()
        torch.testing.assert_close(a, rk[rows], rtol=0, atol=0, equal_nan=True)
        torch.testing.assert_close(c, rv[rows], rtol=0, atol=0, equal_nan=True)


def test_fork_by_hand():
    # pages of 4: row 0 holds 6 tokens in 3, 1, row 1 holds 4 in 0; page 5 is held from elsewhere
    pool = torch.arange(8)[None, :, None].repeat(2, 1, 4)
    table, used, owners = [[3, 1, -1], [0, -1, -1]], [6, 4], [1, 1, 0, 1, 0, 1, 0, 0]
    got = C.fork(pool, table, used, owners, 4, [0, 0, -1, 0], [1, 2, 5, 3])
    # row 1 copies page 1 to 0 (given up by the old row 1); row 2 starts in 2, 4; row 3 copies to 6
    # and needs a page for the ninth token
    assert got == ([[3, 1, -1], [3, 0, -1], [2, 4, -1], [3, 6, 7]], [7, 8, 5, 9],
                   [1, 1, 1, 3, 1, 1, 1, 1], 0)
    assert pool[1, :, 0].tolist() == [1, 1, 2, 3, 4, 5, 1, 7]
    assert C.fork(None, table, used, owners, 4, [0, 0, 0, 0], [9, 9, 9, 9])[3] == (7 - 5) + 4


def test_compact_by_hand():
    pool = torch.arange(7)[None, :, None].clone()
    got = C.compact(pool, [[6, 2, -1], [6, 5, 1]], [0, 1, 1, 0, 0, 1, 2])
    assert got == ([[3, 2, -1], [3, 0, 1]], [1, 1, 1, 2, 0, 0, 0], [-1, 1, 2, -1, -1, 0, 3])
    assert pool[0, :, 0].tolist() == [5, 1, 2, 6, 4, 5, 6]
