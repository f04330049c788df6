"""The operators on 4-bit caches on the GPU against their 64-bit reference."""
import math

import pytest
import torch

import attention_reference as R
import cache_reference as C
from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from modulated_deformable_convolution_amd import cache as K

pytestmark = pytest.mark.gpu
ensure_built()

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def within(got, ref, what):
    value, bound = ref
    got = got.double().cpu()
    same = (got == value) | (got.isnan() & value.isnan())
    bad = ~same & ~((got - value).abs() <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its bound" % (
        what, int(bad.sum()), bad.numel(),
        float(((got - value).abs() / bound.clamp(min=1e-300))[bad].nan_to_num(math.inf).max()))


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def cu(lens):
    c = [0]
    for v in lens:
        c.append(c[-1] + v)
    return c


def layout(lens, page, gen, spare=2, width=None):
    """A table of shuffled pages for sequences of these lengths, on the CPU, and the pages."""
    need = [-(-v // page) for v in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen).tolist()
    width = width or max(need + [1])
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for j in range(n):
            table[b, j] = order.pop()
    return table, pages


def normal(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


# ---------------------------------------------------------------- keys and values

STORE = [
    # heads, dim, page, tokens of each sequence, new ones among them
    (1, 8, 16, [1], [1]),
    (2, 32, 16, [17, 0, 5], [3, 0, 5]),
    (3, 40, 32, [70, 33, 1], [40, 33, 1]),
    (8, 64, 64, [100], [37]),
    (4, 72, 16, [31, 16, 48, 2], [1, 16, 17, 2]),
    (2, 96, 128, [129, 300], [2, 171]),
    (8, 128, 16, [15, 16, 17, 33, 7], [1, 1, 1, 1, 1]),
    (1, 120, 256, [257], [257]),
    (5, 128, 32, [1] * 70 + [40], [1] * 70 + [39]),
]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("case", STORE, ids=str)
def test_store_and_load(case, dt):
    heads, dim, page, lens, new = case
    dtype, gen = DTYPES[dt], torch.Generator().manual_seed(1)
    table, pages = layout(lens, page, gen)
    op = K.mdcn_cache_create(heads, dim, page)
    assert op.page_bytes == C.page_bytes(heads, dim, page)
    pool = torch.randint(0, 256, (pages, op.page_bytes), generator=gen, dtype=torch.uint8)
    kv = normal(gen, sum(new), 2 * heads + 1, dim)
    kv = (kv * torch.exp(3 * normal(gen, sum(new), 2 * heads + 1, 1))).to(dtype)
    k, v = kv[:, :heads], kv[:, heads + 1:]
    dev, there = kv.cuda(), pool.cuda()
    ends = cu(new)
    args = (table.cuda(), ints(lens), ints(ends))
    K.store(op, there, dev[:, :heads], dev[:, heads + 1:], *args)
    C.store(pool, heads, dim, page, k, v, table, lens, ends, dtype)
    # padding channels hold anything; what stands for values must be those bytes
    got = there.cpu()
    for p in range(pages):
        for a, b in zip(C.read_page(got, heads, dim, page, p), C.read_page(pool, heads, dim, page, p)):
            torch.testing.assert_close(a, b, rtol=0, atol=0, equal_nan=True)
    gk, gv = K.load(op, there, *args, sum(new), dtype)
    for a, x in ((gk, k), (gv, v)):
        torch.testing.assert_close(a.cpu().double(), C.rounded(x, dtype), rtol=0, atol=0)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_store_takes_what_is_not_finite_and_the_ends_of_the_range(dt):
    dtype = DTYPES[dt]
    heads, dim, page = 2, 64, 16
    lo, hi = C.LIMITS[dtype]
    top = torch.finfo(dtype).max
    rows = [0.0, -0.0, math.inf, -math.inf, math.nan, top, -top, 2.0 ** (hi + 2), 7 * 2.0 ** (hi - 1),
            7 * 2.0 ** lo, 2.0 ** (lo - 1), 2.0 ** (lo - 2), 1.0, torch.finfo(dtype).smallest_normal,
            torch.finfo(dtype).tiny * torch.finfo(dtype).eps]
    k, v = (normal(torch.Generator().manual_seed(s), len(rows), heads, dim, dtype=dtype) for s in (0, 1))
    for i, x in enumerate(rows):
        (k if i % 2 else v)[i, 1, 33] = min(max(x, -top), top) if abs(x) < math.inf else x
        if abs(x) < 2.0 ** (lo + 4):                  # whole blocks of small values
            for y in (k, v):
                y[i, 1, 32:] = x
                y[i, 1, 40:45] = -x / 2
    op = K.mdcn_cache_create(heads, dim, page)
    pool = torch.full((1, op.page_bytes), 255, dtype=torch.uint8, device="cuda")
    table, used, ends = ints([[0]]), ints([len(rows)]), ints([0, len(rows)])
    K.store(op, pool, k.cuda(), v.cuda(), table, used, ends)
    gk, gv = K.load(op, pool, table, used, ends, len(rows), dtype)
    rk, rv = C.rounded_pair(k, v, dtype)
    assert rk.isnan().any() and rv.isnan().any()
    torch.testing.assert_close(gk.cpu().double(), rk, rtol=0, atol=0, equal_nan=True)
    torch.testing.assert_close(gv.cpu().double(), rv, rtol=0, atol=0, equal_nan=True)


def test_tokens_without_a_page_and_of_no_sequence():
    heads, dim, page = 2, 32, 16
    gen = torch.Generator().manual_seed(5)
    op = K.mdcn_cache_create(heads, dim, page)
    pool = torch.randint(0, 200, (3, op.page_bytes), generator=gen, dtype=torch.uint8)
    table = torch.tensor([[0, -1, 7], [2, 3, -5]], dtype=torch.int32)
    used, ends = [34, 20], [2, 12, 36]               # row 1 has more new tokens than tokens
    k, v = (normal(gen, 40, heads, dim) for _ in range(2))
    there = pool.cuda()
    args = (table.cuda(), ints(used), ints(ends))
    K.store(op, there, k.cuda(), v.cuda(), *args)
    C.store(pool, heads, dim, page, k, v, table, used, ends, torch.float32)
    torch.testing.assert_close(there.cpu(), pool, rtol=0, atol=0)
    gk, gv = K.load(op, there, *args, 40, torch.float32)
    want = torch.zeros(2, 40, heads, dim, dtype=torch.float64)
    for b in range(2):
        n = ends[b + 1] - ends[b]
        x = C.tokens(pool, heads, dim, page, table, b, range(used[b] - n, used[b]))
        want[:, ends[b]:ends[b + 1]] = torch.stack(x[:2])
    torch.testing.assert_close(torch.stack((gk, gv)).cpu().double(), want, rtol=0, atol=0)
    k0, v0 = (torch.full((40, heads, dim), 3.0, device="cuda") for _ in range(2))
    K.load(op, there, *args, 40, torch.float32, k=k0, v=v0)
    given = want.clone()
    given[:, :2] = given[:, 36:] = 3.0
    torch.testing.assert_close(torch.stack((k0, v0)).cpu().double(), given, rtol=0, atol=0)
    k0.fill_(3.0)                                     # one given, the other allocated
    k1, v1 = K.load(op, there, *args, 40, torch.float32, k=k0)
    assert k1 is k0
    torch.testing.assert_close(k0.cpu().double(), given[0], rtol=0, atol=0)
    torch.testing.assert_close(v1.cpu().double(), want[1], rtol=0, atol=0)


# ---------------------------------------------------------------- attention

def filled(gen, heads, dim, page, pages, dtype):
    """A pool on the CPU with a rounded token everywhere."""
    k, v = (normal(gen, pages * page, heads, dim, dtype=dtype) for _ in range(2))
    op = K.mdcn_cache_create(heads, dim, page)
    pool = torch.zeros(pages, op.page_bytes, dtype=torch.uint8, device="cuda")
    table = torch.arange(pages, dtype=torch.int32).cuda()[None]
    n = pages * page
    K.store(op, pool, k.cuda(), v.cuda(), table, ints([n]), ints([0, n]))
    return op, pool.cpu()


def attend_reference(pool, heads, dim, page, table, lens, q, ends, causal, scale, dtype):
    ks, vs = [], []
    for b, n in enumerate(lens):
        k, v, there = C.tokens(pool, heads, dim, page, table, b, range(n))
        assert there.all()
        ks.append(k)
        vs.append(v)
    return R.attend(q, torch.cat(ks), torch.cat(vs), ends, cu(lens), None, causal, scale, dtype)


ATTEND = [
    # q heads, k heads, dim, page, tokens of each sequence, queries of each, causal
    (1, 1, 8, 16, [1], [1], True),
    (4, 2, 32, 16, [1, 17, 300], [1, 1, 1], True),
    (8, 2, 64, 16, [129, 5, 33], [5, 5, 1], True),
    (6, 3, 40, 32, [64, 0, 31, 32], [1, 1, 0, 2], True),
    (7, 1, 72, 64, [200, 90], [3, 7], True),
    (8, 8, 96, 16, [97, 1000], [1, 2], False),
    (32, 8, 128, 16, [2050], [1], True),
    (32, 2, 128, 32, [700, 40], [2, 2], True),
    (16, 4, 80, 32, [333, 64, 5], [5, 5, 5], True),
    (4, 2, 128, 128, [300, 70], [130, 70], True),
    (3, 3, 64, 256, [90, 257], [90, 40], False),
    (2, 1, 56, 16, [20, 33], [25, 40], True),          # more queries than tokens
    (2, 2, 32, 16, [3] * 66 + [100, 0, 9], [1] * 66 + [2, 1, 0], True),
    (64, 1, 128, 16, [130], [1], True),
    (8, 2, 128, 16, [500, 33, 0, 64], [300, 33, 5, 1], True),
    (4, 4, 64, 32, [700, 129], [200, 129], True),
    (12, 2, 96, 64, [257, 1000], [100, 64], False),
    (6, 1, 32, 16, [30, 200], [60, 150], True),        # more queries than tokens
    (2, 1, 80, 128, [1500], [400], True),
]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("case", ATTEND, ids=str)
def test_attend(case, dt):
    hq, hk, dim, page, lens, new, causal = case
    dtype, gen = DTYPES[dt], torch.Generator().manual_seed(2)
    table, pages = layout(lens, page, gen)
    op, pool = filled(gen, hk, dim, page, pages, dtype)
    for b, n in enumerate(lens):                     # what nobody has written yet holds anything
        if n % page:
            spoil(pool, hk, dim, page, int(table[b, n // page]), n % page)
    att = A.mdcn_attention_create(hq, hk, dim, causal)
    q = normal(gen, sum(new), hq + 1, dim, dtype=dtype)
    ends = cu(new)
    dev = q.cuda()[:, 1:]
    args = (pool.cuda(), table.cuda(), ints(lens), ints(ends))
    out, lse = K.attend(att, op, dev, *args)
    ref = attend_reference(pool, hk, dim, page, table, lens, q[:, 1:], ends, causal, att.scale, dtype)
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")
    again = K.attend(att, op, dev, *args)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def spoil(pool, heads, dim, page, p, first):
    k, v, ke, ve, _ = C._place_arrays(heads, dim, page)
    pool[p, k[first:].flatten()] = 0x9e
    pool[p, v[first:].flatten()] = 0x57
    pool[p, ke[first:].flatten()] = 255
    pool[p, ve[first:].flatten()] = 255


@pytest.mark.parametrize("dt", list(DTYPES))
def test_attend_passes_over_missing_pages_and_hidden_nans(dt):
    hq, hk, dim, page, dtype = 4, 2, 64, 16, DTYPES[dt]
    gen = torch.Generator().manual_seed(3)
    op, pool = filled(gen, hk, dim, page, 8, dtype)
    there = pool.cuda()
    table = torch.tensor([[0, -1, 99, 3], [4, 5, 6, 7]], dtype=torch.int32)
    # the last token of row 1 is a NaN in head 1: only the last query sees it
    bad = normal(gen, 1, hk, dim, dtype=dtype)
    bad[0, 1, 3] = math.nan
    K.store(op, there, bad.cuda(), bad.cuda(), ints([[4, 5, 6, 7]]), ints([60]), ints([0, 1]))
    att = A.mdcn_attention_create(hq, hk, dim, True)
    q = normal(gen, 6, hq, dim, dtype=dtype)
    out, lse = K.attend(att, op, q.cuda(), there, table.cuda(), ints([55, 60]), ints([0, 3, 6]))
    pool = there.cpu()
    for b, (n, rows) in enumerate(((55, slice(0, 3)), (60, slice(3, 6)))):
        k, v, held = C.tokens(pool, hk, dim, page, table, b, range(n))
        for i in range(3):
            see = held & (torch.arange(n) <= n - 3 + i)
            r = R.attend(q[rows][i:i + 1], k[see], v[see], [0, 1], [0, int(see.sum())], None, False,
                         att.scale, dtype)
            within(out[rows][i:i + 1], r["out"], "out %d %d" % (b, i))
            nan = lse[:, rows][:, i].isnan().cpu()
            assert nan.tolist() == [False, False] + [b == 1 and i == 2] * 2
            within(lse[:, rows][~nan, i:i + 1], [x[~nan] for x in r["lse"]], "lse %d %d" % (b, i))


def test_attend_rows_of_no_sequence_and_empty_caches():
    att = A.mdcn_attention_create(2, 1, 32, True)
    op = K.mdcn_cache_create(1, 32, 16)
    pool = torch.full((1, op.page_bytes), 255, dtype=torch.uint8, device="cuda")
    q = torch.ones(9, 2, 32, device="cuda")
    for table, used, ends in ((ints([[0], [0]]), ints([0, -3]), ints([2, 5, 7])),
                              (ints([[-1], [5]]), ints([9, 9]), ints([2, 5, 7])),
                              (torch.empty(2, 0, dtype=torch.int32, device="cuda"), ints([4, 4]),
                               ints([2, 5, 7])),
                              (torch.empty(0, 3, dtype=torch.int32, device="cuda"), ints([]), ints([4]))):
        out, lse = K.attend(att, op, q, pool, table, used, ends)
        assert torch.equal(out, torch.zeros_like(q)) and bool((lse == -math.inf).all())
    out, lse = torch.full_like(q, 7.0), torch.full((2, 9), 7.0, device="cuda")
    K.attend(att, op, q, pool, ints([[0], [0]]), ints([0, 0]), ints([2, 5, 7]), out=out, lse=lse)
    inside = torch.zeros(9, dtype=torch.bool)
    inside[2:7] = True
    assert bool((out[inside] == 0).all()) and bool((out[~inside] == 7).all())
    assert bool((lse[:, inside] == -math.inf).all()) and bool((lse[:, ~inside] == 7).all())
    empty = torch.empty(0, op.page_bytes, dtype=torch.uint8, device="cuda")
    out, lse = K.attend(att, op, q, empty, ints([[0], [0]]), ints([3, 3]), ints([0, 5, 9]))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


# ---------------------------------------------------------------- pages

FORK = [
    # rows in, rows out, width, page tokens, pages, layers, page bytes, seed
    (1, 1, 4, 16, 6, 1, 544, 0),
    (4, 8, 9, 16, 80, 2, 1088, 1),
    (32, 32, 40, 16, 900, 1, 2176, 2),
    (5, 3, 7, 32, 50, 3, 48, 3),
    (40, 130, 30, 64, 3000, 1, 16, 4),
    (300, 300, 300, 4, 40000, 1, 16, 5),              # more than one workgroup's bookkeeping
    (7, 6, 3, 10, 17, 2, 40000, 6),                   # not enough pages
]


def fork_case(case):
    rows, out, width, page, pages, layers, size, seed = case
    g = torch.Generator().manual_seed(seed)
    ri = lambda hi, *n: torch.randint(0, hi, n, generator=g)  # noqa: E731
    order = torch.randperm(pages, generator=g).tolist()
    table, used, owners = [], [], [0] * pages
    for b in range(rows):
        n = int(ri(max(1, (width - 3) * page + 1), 1)) if pages > rows * width else int(ri(2 * page, 1))
        held = -(-n // page)
        row = [order.pop() for _ in range(held)]
        if b and n // page and table[-1][0] >= 0 and used[-1] >= page:
            row[0] = table[-1][0]                     # a shared first page
        if held > 2:
            row[1] = [-1, pages, row[1], row[1]][int(ri(4, 1))]
        row += [-1] * (width - held)
        if held < width and int(ri(3, 1)) == 0 and order:
            row[held] = order.pop()                   # room that was given and not used
        table.append(row)
        used.append(n)
    for row in table:
        for p in row:
            if 0 <= p < pages:
                owners[p] += 1
    owners[order[0]] += 1                             # held from elsewhere
    parents = (ri(rows + 2, out) - 1).tolist()
    new = (ri(3 * page, out) - 2).tolist()
    pool = torch.randint(0, 256, (layers, pages, size), generator=g, dtype=torch.uint8)
    return pool, table, used, owners, page, parents, new


@pytest.mark.parametrize("which", ["both", "parents", "new"])
@pytest.mark.parametrize("case", FORK, ids=str)
def test_fork(case, which):
    pool, table, used, owners, page, parents, new = fork_case(case)
    if which == "new":
        parents, new = None, (new * len(table))[:len(table)]
    if which == "parents":
        new = None
    there = pool.cuda()
    got = K.fork_pages(there, ints(table), ints(used), ints(owners), page,
                       None if parents is None else ints(parents), None if new is None else ints(new))
    want = C.fork(pool, table, used, owners, page, parents, new)
    assert int(got[3]) == want[3]
    if which == "both":
        assert (want[3] > 0) == (case == FORK[-1])
    for a, b, what in zip(got, want, ("table", "used", "owners")):
        assert a.tolist() == b, what
    assert torch.equal(there.cpu(), pool)


def test_fork_of_nothing_and_without_a_pool():
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    t, u, o, m = K.fork_pages(None, none, ints([]), ints([0, 0, 1, 0]), 16, ints([-1, 5]), ints([17, 3]))
    assert t.tolist() == [[0, 1, -1], [3, -1, -1]] and u.tolist() == [17, 3]
    assert o.tolist() == [1, 1, 1, 1] and m.tolist() == [0]
    t, u, o, m = K.fork_pages(None, none, ints([]), ints([]), 16, ints([]), None)
    assert t.shape == (0, 3) and m.tolist() == [0]


COMPACT = [
    # pages, held, rows, width, layers, page bytes, seed
    (1, 0, 1, 1, 1, 16, 0), (1, 1, 1, 1, 1, 16, 1), (64, 20, 5, 6, 2, 1088, 2), (64, 64, 5, 13, 1, 16, 3),
    (1024, 600, 30, 25, 1, 48, 4), (1025, 1024, 30, 40, 1, 48, 5), (5000, 1, 1, 2, 1, 32, 6),
    (70001, 33333, 600, 120, 1, 16, 7), (300, 150, 10, 15, 3, 17408, 8),
]


@pytest.mark.parametrize("case", COMPACT, ids=str)
def test_compact(case):
    pages, held, rows, width, layers, size, seed = case
    g = torch.Generator().manual_seed(seed)
    owners = torch.zeros(pages, dtype=torch.int32)
    owners[torch.randperm(pages, generator=g)[:held]] = \
        torch.randint(1, 4, (held,), generator=g).to(torch.int32)
    if held < pages:
        owners[int((owners == 0).nonzero()[0])] = -2
    table = torch.randint(-2, pages + 2, (rows, width), generator=g).to(torch.int32)
    pool = torch.randint(0, 256, (layers, pages, size), generator=g, dtype=torch.uint8)
    there = pool.cuda()
    got = K.compact_pages(there, table.cuda(), owners.cuda())
    want = C.compact(pool, table.tolist(), owners.tolist())
    for a, b, what in zip(got, want, ("table", "owners", "moved")):
        assert a.tolist() == b, what
    assert torch.equal(there.cpu(), pool)


@pytest.mark.parametrize("layers,count,size", [(1, 1, 16), (3, 7, 544), (2, 20, 16384 * 2 + 48), (1, 0, 16)])
def test_copy(layers, count, size):
    g = torch.Generator().manual_seed(9)
    a = torch.randint(0, 256, (layers, 30, size), generator=g, dtype=torch.uint8)
    b = torch.randint(0, 256, (layers, 25, size), generator=g, dtype=torch.uint8)
    src = torch.randperm(30, generator=g)[:count]
    dst = torch.randperm(25, generator=g)[:count]
    there = b.cuda()
    odd = torch.tensor([-1, 30, 3, 4], dtype=torch.int32)
    K.copy_pages(a.cuda(), there, torch.cat((src.to(torch.int32), odd)).cuda(),
                 torch.cat((dst.to(torch.int32), torch.tensor([1, 2, -1, 25], dtype=torch.int32))).cuda())
    b[:, dst] = a[:, src]
    assert torch.equal(there.cpu(), b)
    pool = a.cuda()[:, :25]                           # within one pool, pages of a larger one
    K.copy_pages(pool, pool, ints([3, 4]), ints([5, 6]))
    want = a[:, :25].clone()
    want[:, 5:7] = want[:, 3:5]
    assert torch.equal(pool.cpu(), want)
    flat = a[0].cuda()                                # and to pages past those of a part of it
    K.copy_pages(flat[:5], flat, ints([2, 4]), ints([29, 9]))
    want = a[0].clone()
    want[29], want[9] = a[0][2], a[0][4]
    assert torch.equal(flat.cpu(), want)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_many_queries_pass_over_missing_pages_and_hidden_nans(dt):
    hq, hk, dim, page, dtype, new = 4, 2, 40, 16, DTYPES[dt], 90
    gen = torch.Generator().manual_seed(21)
    op, pool = filled(gen, hk, dim, page, 12, dtype)
    there, n = pool.cuda(), 170
    table = torch.tensor([[0, 1, -1, 3, 12, 5, 6, -9, 8, 9, 10]], dtype=torch.int32)
    bad = normal(gen, 1, hk, dim, dtype=dtype)        # token 150 is a NaN in head 0
    bad[0, 0, 17] = math.nan
    K.store(op, there, bad.cuda(), bad.cuda(), table.cuda(), ints([151]), ints([0, 1]))
    att = A.mdcn_attention_create(hq, hk, dim, True)
    assert K.describe_attend(att, op, dtype, 1, new, 11).startswith("tile")
    q = normal(gen, new, hq, dim, dtype=dtype)
    out, lse = K.attend(att, op, q.cuda(), there, table.cuda(), ints([n]), ints([0, new]))
    k, v, held = C.tokens(there.cpu(), hk, dim, page, table, 0, range(n))
    out, lse = out.cpu(), lse.cpu()
    for i in range(new):
        see = held & (torch.arange(n) <= n - new + i)
        r = R.attend(q[i:i + 1], k[see], v[see], [0, 1], [0, int(see.sum())], None, False, att.scale, dtype)
        within(out[i:i + 1], r["out"], "out %d" % i)
        nan = [n - new + i >= 150] * 2 + [False] * 2
        assert lse[:, i].isnan().tolist() == nan
        within(lse[2:, i:i + 1], [x[2:] for x in r["lse"]], "lse %d" % i)
