"""The operators on 4-bit caches on the GPU: layouts, streams, graphs, sizes past 32 bits and
a run of all of them together."""
import math

import pytest
import torch

import attention_reference as R
import cache_reference as C
from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from modulated_deformable_convolution_amd import cache as K
from test_gpu_cache import (DTYPES, attend_reference, cu, filled, ints, layout, normal, within)

pytestmark = pytest.mark.gpu
ensure_built()


# every kernel: types, blocks of channels and rows of a workgroup
@pytest.mark.parametrize("dim", [24, 64, 88, 128])
@pytest.mark.parametrize("new,shape", [(2, "split rows=16"), (12, "split rows=32"), (70, "tile")])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_every_kernel(dt, new, shape, dim):
    dtype, gen, lens = DTYPES[dt], torch.Generator().manual_seed(11), [333, 150]
    table, pages = layout(lens, 32, gen)
    op, pool = filled(gen, 2, dim, 32, pages, dtype)
    att = A.mdcn_attention_create(4, 2, dim, True)
    if dt == "f32" and new == 12:                      # up to 64 rows in tiles of 16
        shape = "split rows=16"
    assert K.describe_attend(att, op, dtype, 2, 2 * new, table.shape[1]).startswith(shape)
    q = normal(gen, 2 * new, 4, dim, dtype=dtype)
    out, lse = K.attend(att, op, q.cuda(), pool.cuda(), table.cuda(), ints(lens), ints([0, new, 2 * new]))
    ref = attend_reference(pool, 2, dim, 32, table, lens, q, [0, new, 2 * new], True, att.scale, dtype)
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")


@pytest.mark.parametrize("new", [1, 130])
def test_hundreds_of_sequences(new):
    gen, n = torch.Generator().manual_seed(12), 150
    lens = [(37 * i) % 90 + new for i in range(n)]
    rows = [new if i % 3 else 0 for i in range(n)]
    table, pages = layout(lens, 16, gen)
    op, pool = filled(gen, 1, 32, 16, pages, torch.float16)
    att = A.mdcn_attention_create(2, 1, 32, True)
    q = normal(gen, sum(rows), 2, 32, dtype=torch.float16)
    out, lse = K.attend(att, op, q.cuda(), pool.cuda(), table.cuda(), ints(lens), ints(cu(rows)))
    ref = attend_reference(pool, 1, 32, 16, table, lens, q, cu(rows), True, att.scale, torch.float16)
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")


def test_layouts_of_pools_and_tables():
    """Layers within pages, rows of a wider table, sequences that share pages or name one twice."""
    gen, heads, dim, page, dtype = torch.Generator().manual_seed(13), 2, 64, 16, torch.bfloat16
    op, flat = filled(gen, heads, dim, page, 7, dtype)
    pool = torch.zeros(7, 3, op.page_bytes, dtype=torch.uint8, device="cuda")
    pool[:, 1] = flat.cuda()
    wide = torch.tensor([[0, 1, 2, 9, 9], [0, 1, 3, 9, 9], [5, 5, 5, 9, 9]], dtype=torch.int32)
    table, lens, rows = wide[:, :3], [40, 37, 48], [1, 2, 1]
    att = A.mdcn_attention_create(4, heads, dim, True)
    q = normal(gen, 4, 4, dim, dtype=dtype)
    args = (pool[:, 1], wide.cuda()[:, :3], ints(lens))
    out, lse = K.attend(att, op, q.cuda(), *args, ints(cu(rows)))
    ref = attend_reference(flat, heads, dim, page, table, lens, q, cu(rows), True, att.scale, dtype)
    within(out, ref["out"], "out")
    k, v = K.load(op, *args, ints([0, 40, 40, 60]), 60, dtype)
    for b, places, at in ((0, range(40), slice(0, 40)), (2, range(28, 48), slice(40, 60))):
        x = C.tokens(flat, heads, dim, page, table, b, places)
        assert torch.equal(k[at].cpu().double(), x[0]) and torch.equal(v[at].cpu().double(), x[1])
    new = normal(gen, 3, 3, heads, dim, dtype=dtype).cuda()          # strides of their own
    K.store(op, pool[:, 1], new[:, 0], new[:, 1], wide.cuda()[:, :3], ints([40, 37, 48]), ints([0, 1, 2, 2]))
    C.store(flat, heads, dim, page, new[:, 0].cpu(), new[:, 1].cpu(), table, [40, 37, 48], [0, 1, 2, 2], dtype)
    assert torch.equal(pool[:, 1].cpu(), flat) and not pool[:, 0].any() and not pool[:, 2].any()


def test_a_pool_of_more_than_4_gib():
    heads, dim, page, dtype = 4, 128, 64, torch.float16
    op = K.mdcn_cache_create(heads, dim, page)
    pages = (5 << 30) // op.page_bytes
    pool = torch.empty(pages, op.page_bytes, dtype=torch.uint8, device="cuda")
    gen = torch.Generator().manual_seed(14)
    table = torch.tensor([[pages - 1, 3, pages - 70], [pages // 2 + 1, pages - 2, 0]], dtype=torch.int32)
    lens = [150, 190]
    k, v = (normal(gen, sum(lens), heads, dim, dtype=dtype) for _ in range(2))
    args = (table.cuda(), ints(lens))
    K.store(op, pool, k.cuda(), v.cuda(), *args, ints(cu(lens)))
    gk, gv = K.load(op, pool, *args, ints(cu(lens)), sum(lens), dtype)
    rk, rv = C.rounded(k, dtype), C.rounded(v, dtype)
    assert torch.equal(gk.cpu().double(), rk) and torch.equal(gv.cpu().double(), rv)
    for new in (1, 70):
        att = A.mdcn_attention_create(8, heads, dim, True)
        q = normal(gen, 2 * new, 8, dim, dtype=dtype)
        out, lse = K.attend(att, op, q.cuda(), pool, *args, ints([0, new, 2 * new]))
        ref = R.attend(q, rk, rv, [0, new, 2 * new], cu(lens), None, True, att.scale, dtype)
        within(out, ref["out"], "out")
        within(lse, ref["lse"], "lse")
    K.copy_pages(pool, pool, ints([pages - 1]), ints([pages // 2 + 9]))
    assert torch.equal(pool[pages // 2 + 9], pool[pages - 1])


@pytest.mark.parametrize("new", [1, 140])
def test_tables_with_room_for_more_units_than_31_bits(new):
    gen, heads, dim, page, dtype = torch.Generator().manual_seed(15), 64, 8, 256, torch.bfloat16
    lens = [700, 300, 1, 0, 64, 65, 257, 512]
    table, pages = layout(lens, page, gen)
    width = 1 << 20
    room = torch.full((8, width), -1, dtype=torch.int32, device="cuda")
    room[:, :table.shape[1]] = table.cuda()
    op, pool = filled(gen, heads, dim, page, pages, dtype)
    att = A.mdcn_attention_create(heads, heads, dim, False)
    assert int(K.describe_attend(att, op, dtype, 8, 8 * new, width).split("=")[-1]) > 64
    q = normal(gen, 8 * new, heads, dim, dtype=dtype)
    ends = [i * new for i in range(9)]
    out, lse = K.attend(att, op, q.cuda(), pool.cuda(), room, ints(lens), ints(ends))
    ref = attend_reference(pool, heads, dim, page, table, lens, q, ends, False, att.scale, dtype)
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_ends_of_the_range_and_queries_that_are_not_finite(dt, new):
    dtype, heads, dim, page = DTYPES[dt], 1, 64, 16
    gen = torch.Generator().manual_seed(16)
    lo, hi = C.LIMITS[dtype]
    n = 100
    k, v = (normal(gen, n, heads, dim) for _ in range(2))
    scale = 2.0 ** torch.tensor([0, lo + 1, hi - 2, 0, -3] * 20)[:n].double()
    k[:, :, 32:] *= 2.0 ** -8                          # blocks of different exponents
    v = (v.double() * scale[:, None, None]).to(dtype)
    k = k.to(dtype)
    op = K.mdcn_cache_create(heads, dim, page)
    table = torch.arange(7, dtype=torch.int32)[None]
    pool = torch.zeros(7, op.page_bytes, dtype=torch.uint8, device="cuda")
    K.store(op, pool, k.cuda(), v.cuda(), table.cuda(), ints([n]), ints([0, n]))
    rk, rv = C.rounded(k, dtype), C.rounded(v, dtype)
    att = A.mdcn_attention_create(2, heads, dim, True)
    q = normal(gen, new + 2, 2, dim, dtype=dtype)
    q[-2, 0, 5] = math.inf
    q[-1, 1, 40] = math.nan
    out, lse = K.attend(att, op, q.cuda(), pool, table.cuda(), ints([n]), ints([0, new + 2]))
    ref = R.attend(torch.nan_to_num(q, 0, 0, 0), rk, rv, [0, new + 2], [0, n], None, True, att.scale, dtype)
    bad = torch.zeros(new + 2, 2, dtype=torch.bool)
    bad[-2, 0] = bad[-1, 1] = True
    assert bool(out.cpu()[bad].isnan().all()) and bool(lse.t().cpu()[bad].isnan().all())
    value, bound = (x[~bad] for x in ref["out"])
    # a value that rounds past the type's largest one becomes infinite, on both sides alike
    within(out.cpu()[~bad], (value.to(dtype).double() if dt != "f32" else value, bound), "out")
    within(lse.t().cpu()[~bad], [x.t()[~bad] for x in ref["lse"]], "lse")


def test_offsets_and_lengths_out_of_range_are_clamped():
    gen, dtype = torch.Generator().manual_seed(17), torch.float32
    op, pool = filled(gen, 1, 32, 16, 4, dtype)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    att = A.mdcn_attention_create(1, 1, 32, True)
    q = normal(gen, 6, 1, 32, dtype=dtype)
    out, lse = K.attend(att, op, q.cuda(), pool.cuda(), table.cuda(), ints([1 << 30, 20]), ints([-9, 4, 99]))
    ref = attend_reference(pool, 1, 32, 16, table, [32, 20], q, [0, 4, 6], True, att.scale, dtype)
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")
    there, k = pool.cuda(), normal(gen, 6, 1, 32)
    K.store(op, there, k.cuda(), k.cuda(), table.cuda(), ints([5, 20]), ints([-9, 4, 99]))
    C.store(pool, 1, 32, 16, k, k, table, [5, 20], [0, 4, 6], dtype)
    assert torch.equal(there.cpu(), pool)
    for ends in ([5, 2, 4], [6, 6, 0], [3, 99, -7]):   # whatever they mean, nothing is out of bounds
        K.attend(att, op, q.cuda(), there, table.cuda(), ints([32, 20]), ints(ends))
        K.load(op, there, table.cuda(), ints([32, 20]), ints(ends), 6, dtype)
        K.store(op, there, k.cuda(), k.cuda(), table.cuda(), ints([32, 20]), ints(ends))
    torch.cuda.synchronize()


# ---------------------------------------------------------------- pages

def test_fork_and_compact_of_thousands_of_rows():
    g = torch.Generator().manual_seed(18)
    rows, page, pages = 2500, 16, 20000
    order = torch.randperm(pages, generator=g).tolist()
    used = torch.randint(0, 49, (rows,), generator=g).tolist()
    table = [[order.pop() if j * page < n else -1 for j in range(4)] for n in used]
    owners = [0] * pages
    for row in table:
        for p in row:
            if p >= 0:
                owners[p] += 1
    parents = torch.randint(-1, rows, (2300,), generator=g).tolist()
    new = torch.randint(0, 3, (2300,), generator=g).tolist()
    pool = torch.randint(0, 256, (2, pages, 32), generator=g, dtype=torch.uint8)
    there = pool.cuda()
    got = K.fork_pages(there, ints(table), ints(used), ints(owners), page, ints(parents), ints(new))
    want = C.fork(pool, table, used, owners, page, parents, new)
    assert int(got[3]) == want[3] == 0
    for a, b in zip(got, want):
        assert a.flatten().tolist() == torch.tensor(b).flatten().tolist()
    assert torch.equal(there.cpu(), pool)
    got = K.compact_pages(there, got[0], got[2])
    want = C.compact(pool, want[0], want[2])
    for a, b in zip(got, want):
        assert a.flatten().tolist() == torch.tensor(b).flatten().tolist()
    assert torch.equal(there.cpu(), pool)


def test_results_that_the_caller_gives():
    table, used, owners = ints([[1, -1], [0, -1]]), ints([5, 9]), ints([1, 1, 0, 0, 0])
    pool = torch.zeros(1, 5, 16, dtype=torch.uint8, device="cuda")
    out = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((2, 2), (2,), (5,), (1,))]
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    got = K.fork_pages(pool, table, used, owners, 16, ints([0, 0]), ints([1, 20]), *out, workspace=ws)
    assert all(a is b for a, b in zip(got, out))
    assert [x.tolist() for x in out] == [[[1, -1], [0, 2]], [6, 25], [1, 1, 1, 0, 0], [0]]
    out = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((2, 2), (5,), (5,))]
    K.compact_pages(pool, ints([[4, -1], [2, 4]]), ints([0, 0, 1, 0, 2]), *out, workspace=ws)
    assert [x.tolist() for x in out] == [[[1, -1], [0, 1]], [1, 2, 0, 0, 0], [-1, -1, 0, -1, 1]]


# ---------------------------------------------------------------- streams and graphs

def decode_state(dtype=torch.bfloat16, lens=(30, 17, 64, 5)):
    gen = torch.Generator().manual_seed(19)
    heads, dim, page = 2, 64, 16
    table, pages = layout(list(lens), page, gen, spare=40, width=40)
    op, pool = filled(gen, heads, dim, page, pages, dtype)
    owners = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    att = A.mdcn_attention_create(4, heads, dim, True)
    return gen, op, att, pool, table, ints(list(lens)), owners


def step(op, att, pool, table, used, owners, parents, k, v, q, stream=None):
    n = q.shape[0]
    ends = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    ones = torch.ones(n, dtype=torch.int32, device="cuda")
    if stream:
        torch.cuda.current_stream().synchronize()     # what the call reads is there
    t, u, o, m = K.fork_pages(pool, table, used, owners, op.page, parents, ones, stream=stream)
    K.store(op, pool, k, v, t, u, ends, stream=stream)
    out, lse = K.attend(att, op, q, pool, t, u, ends, stream=stream)
    return t, u, o, m, out, lse


def test_a_captured_step_is_replayed():
    gen, op, att, pool, table, used, owners = decode_state()
    table, owners = table.cuda(), owners.cuda()
    make = lambda *s: normal(gen, *s, dtype=torch.bfloat16).cuda()  # noqa: E731
    x = dict(k=make(4, 2, 64), v=make(4, 2, 64), q=make(4, 4, 64), parents=ints([0, 1, 2, 3]))
    mine = pool.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(op, att, mine.clone(), table, used, owners, **x)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(op, att, mine, table, used, owners, **x)
        more = step(op, att, mine, got[0], got[1], got[2], **x)         # a workspace of its own
    for parents in ([0, 1, 2, 3], [1, 1, 0, -1], [3, 3, 3, 3], [2, 0, 2, 1]):
        mine.copy_(pool)
        x["parents"].copy_(ints(parents))
        for n in ("k", "v", "q"):
            x[n].copy_(make(*x[n].shape))
        graph.replay()
        torch.cuda.synchronize()
        other = pool.cuda()
        want = step(op, att, other, table, used, owners, **x)
        want2 = step(op, att, other, want[0], want[1], want[2], **x)
        for a, b in zip(got + more, want + want2):
            assert torch.equal(a, b)
        assert torch.equal(mine, other)


def test_two_calls_on_two_streams():
    states, streams, results = [], [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        gen, op, att, pool, table, used, owners = decode_state(lens=(500 + i, 17, 64, 5))
        make = lambda *s: normal(gen, *s, dtype=torch.bfloat16).cuda()  # noqa: E731
        states.append((op, att, pool.cuda(), table.cuda(), used, owners.cuda(), ints([0, 0, 2, 1]),
                       make(4, 2, 64), make(4, 2, 64), make(4, 4, 64)))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x in zip(streams, states):
            pool = x[2].clone()
            torch.cuda.synchronize()
            results.append((x, pool, step(x[0], x[1], pool, *x[3:], stream=s.cuda_stream)))
    torch.cuda.synchronize()
    for x, pool, got in results:
        other = x[2].clone()
        want = step(x[0], x[1], other, *x[3:])
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(pool, other)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dt", list(DTYPES))
def test_beams_decode_as_their_own_sequences(dt):
    """Beams that fork, share pages, are compacted, swapped out and in again attend as sequences
    whose rounded keys and values are kept one by one."""
    dtype, heads, dim, page, layers = DTYPES[dt], 2, 40, 16, 2
    gen = torch.Generator().manual_seed(20)
    op = K.mdcn_cache_create(heads, dim, page)
    att = A.mdcn_attention_create(4, heads, dim, True)
    pool = torch.randint(0, 256, (layers, 64, op.page_bytes), generator=gen, dtype=torch.uint8).cuda()
    table = torch.full((0, 6), -1, dtype=torch.int32, device="cuda")
    used, owners = ints([]), torch.zeros(64, dtype=torch.int32, device="cuda")
    kept = []                                        # per row: rounded (k, v) of each layer
    prompt, n = [20, 33, 1, 7], 4
    plan = [([-1] * 4, prompt), ([0, 0, 1, 3, 3], None), ([4, 2, 2, 0, 1, 1], None), ([5, 4, 3, 0, 0], None),
            ([0, 1, 2, 4, 4, 4, 2], None), ([6, 5, 1, 0], None), ([3, 3, 2, 1, -1], None)]
    for turn, (parents, new) in enumerate(plan):
        new = new or [1 + (turn + i) % 3 for i in range(len(parents))]
        table, used, owners, missing = K.fork_pages(pool, table, used, owners, page, ints(parents),
                                                    ints(new))
        assert int(missing) == 0
        n, ends = sum(new), cu(new)
        kept = [[(x[0].clone(), x[1].clone()) for x in kept[p]] if p >= 0 else
                [(torch.zeros(0, heads, dim).double(),) * 2] * layers for p in parents]
        for layer in range(layers):
            k, v = (normal(gen, n, heads, dim, dtype=dtype) for _ in range(2))
            q = normal(gen, n, 4, dim, dtype=dtype)
            K.store(op, pool[layer], k.cuda(), v.cuda(), table, used, ints(ends))
            rk, rv = C.rounded(k, dtype), C.rounded(v, dtype)
            for i in range(len(parents)):
                s = slice(ends[i], ends[i + 1])
                kept[i][layer] = tuple(torch.cat((a, b[s])) for a, b in zip(kept[i][layer], (rk, rv)))
            out, lse = K.attend(att, op, q.cuda(), pool[layer], table, used, ints(ends))
            lens = [x[layer][0].shape[0] for x in kept]
            assert used.tolist() == lens
            ref = R.attend(q, *(torch.cat([x[layer][i] for x in kept]) for i in range(2)), ends, cu(lens),
                           None, True, att.scale, dtype)
            within(out, ref["out"], "out of turn %d" % turn)
            within(lse, ref["lse"], "lse of turn %d" % turn)
        held = sorted(set(p for row in table.tolist() for p in row if p >= 0))
        assert [i for i, c in enumerate(owners.tolist()) if c] == held
        if turn % 2:
            table, owners, moved = K.compact_pages(pool, table, owners)
            assert [i for i, c in enumerate(owners.tolist()) if c] == list(range(len(held)))
        else:                                        # out to another pool, and back to other pages
            other = torch.empty_like(pool)
            there = ints(held)
            K.copy_pages(pool, other, there, there)
            pool.fill_(255)
            places = torch.randperm(64, generator=gen)[:len(held)].to(torch.int32)
            K.copy_pages(other, pool, there, places.cuda())
            number = torch.full((65,), -1, dtype=torch.int32)
            number[held] = places
            table = number[table.cpu().long()].cuda()
            owners = torch.zeros(64, dtype=torch.int32).index_add(
                0, table[table >= 0].cpu().long(), torch.ones(int((table >= 0).sum()), dtype=torch.int32)).cuda()
