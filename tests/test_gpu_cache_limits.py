"""Attention on 4-bit caches at the ends of what it takes, on the GPU against the 64-bit reference."""
import math

import pytest
import torch

import attention_reference as R
import cache_reference as C
from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from modulated_deformable_convolution_amd import cache as K
from test_gpu_cache import DTYPES, cu, ints, layout, normal, within

pytestmark = pytest.mark.gpu
ensure_built()


def rounded_cache(k, v, lens, page, dtype, gen):
    """A cache of k and v [tokens, heads, dim]: (handle, pool, table), and its values in 64 bits."""
    heads, dim = k.shape[1:]
    op = K.mdcn_cache_create(heads, dim, page)
    table, pages = layout(lens, page, gen)
    pool = torch.full((pages, op.page_bytes), 255, dtype=torch.uint8, device="cuda")
    K.store(op, pool, k.cuda(), v.cuda(), table.cuda(), ints(lens), ints(cu(lens)))
    return op, pool, table.cuda(), C.rounded(k, dtype), C.rounded(v, dtype)


# ---------------------------------------------------------------- more queries than tokens

@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("hq,hk,lens,new", [
    (4, 2, [100, 5, 0, 130], [2500, 700, 300, 64]), (3, 1, [513], [4000]), (8, 8, [1, 64, 65], [900] * 3),
], ids=str)
def test_more_queries_than_tokens(dt, hq, hk, lens, new):
    dtype, gen, dim, page = DTYPES[dt], torch.Generator().manual_seed(31), 40, 32
    k, v = (normal(gen, sum(lens), hk, dim, dtype=dtype) for _ in range(2))
    op, pool, table, rk, rv = rounded_cache(k, v, lens, page, dtype, gen)
    att = A.mdcn_attention_create(hq, hk, dim, True)
    assert K.describe_attend(att, op, dtype, len(lens), sum(new), table.shape[1]).startswith("tile")
    q = normal(gen, sum(new), hq, dim, dtype=dtype)
    out, lse = K.attend(att, op, q.cuda(), pool, table, ints(lens), ints(cu(new)))
    ref = R.attend(q, rk, rv, cu(new), cu(lens), None, True, att.scale, dtype)
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")


@pytest.mark.parametrize("dt,heads", [("bf16", 32), ("f32", 16)])
def test_a_million_queries_before_a_short_cache(dt, heads):
    """Work counted by what queries would see, were there tokens for all, passes 31 bits."""
    dtype, gen, dim, n, new = DTYPES[dt], torch.Generator().manual_seed(32), 8, 100, 1 << 20
    k, v = (normal(gen, n, heads, dim, dtype=dtype) for _ in range(2))
    op, pool, table, rk, rv = rounded_cache(k, v, [n], 16, dtype, gen)
    att = A.mdcn_attention_create(heads, heads, dim, True)
    q = normal(gen, n, heads, dim, dtype=dtype)
    all_q = torch.ones(new, heads, dim, dtype=dtype, device="cuda")
    all_q[-n:] = q.cuda()
    out, lse = K.attend(att, op, all_q, pool, table, ints([n]), ints([0, new]))
    assert not out[:-n].any() and bool((lse[:, :-n] == -math.inf).all())
    ref = R.attend(q, rk, rv, [0, n], [0, n], None, True, att.scale, dtype)
    within(out[-n:], ref["out"], "out")
    within(lse[:, -n:], ref["lse"], "lse")


# what values are: all at the largest one, of both signs, large ones behind a low first score
LARGE = ["equal", "signs", "late"]


@pytest.mark.parametrize("lens,new,causal", [
    ([2], 1, False), ([40, 3], 1, True), ([3000, 1], 2, True),                 # few rows, joined parts
    ([33, 64], 20, False), ([70, 5], 5, True),                                 # two row tiles
    ([200, 70], 70, True), ([1500], 300, True), ([700], 150, False),           # many rows
], ids=str)
@pytest.mark.parametrize("kind", LARGE)
@pytest.mark.parametrize("dim", [32, 96, 128])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_sums_of_values_near_the_largest(dt, dim, kind, lens, new, causal):
    """The mean of values that the format holds is within the type's range, and so is out; a block
    of small values beside them stays exact."""
    dtype, gen, heads = DTYPES[dt], torch.Generator().manual_seed(30), 2
    hi = C.LIMITS[dtype][1]
    n = sum(lens)
    k, v = (normal(gen, n, heads, dim) for _ in range(2))
    q = normal(gen, new * len(lens), 4, dim, dtype=dtype)
    if kind == "late":                               # from token 32 on 7 bits above those before
        q = torch.ones_like(q)
        k = torch.zeros_like(k)
        at = torch.cat([torch.arange(x) for x in lens])
        k[at >= 32] = 1.0
        v = v.clamp(-1, 1) * 2.0 ** (hi - 2)
    else:                                            # infinities are held as the largest value
        k *= 2.0 ** -6
        v = torch.full_like(v, math.inf)
        if kind == "signs":
            v[torch.rand(v.shape, generator=gen) < 0.5] = -math.inf
    if dim > 32:                                     # one block of small values
        v[..., 32:64] = normal(gen, n, heads, 32) * 2.0 ** (C.LIMITS[dtype][0] + 12)
    k, v = k.to(dtype), v.to(dtype)
    op, pool, table, rk, rv = rounded_cache(k, v, lens, 16, dtype, gen)
    scale = 7 * math.log(2) / dim if kind == "late" else None
    att = A.mdcn_attention_create(4, heads, dim, causal, scale)
    ends = [new * i for i in range(len(lens) + 1)]
    out, lse = K.attend(att, op, q.cuda(), pool, table, ints(lens), ints(ends))
    ref = R.attend(q, rk, rv, ends, cu(lens), None, causal, att.scale, dtype)
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")
    again = K.attend(att, op, q.cuda(), pool, table, ints(lens), ints(ends))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("new", [1, 12, 60])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_some_of_many_sequences_hold_values_near_the_largest(dt, new):
    """Among ordinary ones, with a page missing, and where a graph replays the call."""
    dtype, gen, heads, dim, page, n = DTYPES[dt], torch.Generator().manual_seed(33), 2, 64, 16, 130
    lens = [new + (37 * i) % 60 for i in range(n)]
    k, v = (normal(gen, sum(lens), heads, dim) for _ in range(2))
    for b in range(0, n, 3):
        v[sum(lens[:b]):sum(lens[:b + 1]), b % 2, 32 * (b % 2):] = math.inf
    k, v = k.to(dtype), v.to(dtype)
    op, pool, table, rk, rv = rounded_cache(k, v, lens, page, dtype, gen)
    table[3, 0] = -1                                  # row 3 begins with token 16
    keys, values, held = [], [], []
    for b in range(n):
        s = slice(sum(lens[:b]) + (16 if b == 3 else 0), sum(lens[:b + 1]))
        keys.append(rk[s])
        values.append(rv[s])
        held.append(max(lens[b] - 16, 0) if b == 3 else lens[b])
    att = A.mdcn_attention_create(2, heads, dim, True)
    ends = [new * i for i in range(n + 1)]
    q = normal(gen, new * n, 2, dim, dtype=dtype)
    ref = R.attend(q, torch.cat(keys), torch.cat(values), ends, cu(held), None, True, att.scale, dtype)
    args = (q.cuda(), pool, table, ints(lens), ints(ends))
    out, lse = K.attend(att, op, *args)
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        K.attend(att, op, *args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = K.attend(att, op, *args)
    for _ in range(3):
        got[0].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        assert torch.equal(K.attend(att, op, *args)[0], out)


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_values_near_the_largest_leave_the_other_rows_as_they_were(dt, new):
    """Bit for bit, where their scores are very large too."""
    dtype, gen, heads, dim, page, n = DTYPES[dt], torch.Generator().manual_seed(34), 2, 32, 16, 40
    size = 2.0 ** (60 if dt == "f32" else 12)
    lens = [new + (37 * i) % 60 for i in range(n)]
    k, v = (normal(gen, sum(lens), heads, dim) for _ in range(2))
    k[-lens[-1]:] *= size                             # of the last one
    large = v.clone()
    large[:lens[0]] = math.inf
    q = normal(gen, new * n, 2, dim, dtype=dtype)
    q[-new:] *= size
    att, got = A.mdcn_attention_create(2, heads, dim, True), []
    for x in (v, large):
        op, pool, table, _, _ = rounded_cache(k.to(dtype), x.to(dtype), lens, page, dtype,
                                              torch.Generator().manual_seed(1))
        got.append(K.attend(att, op, q.cuda(), pool, table, ints(lens), ints([new * i for i in range(n + 1)])))
    top = float(C.rounded(large[:1, :, :1].to(dtype), dtype).max())
    assert torch.equal(got[0][0][new:], got[1][0][new:]) and torch.equal(got[0][1], got[1][1])
    assert float((got[1][0][:new].double().cpu() / top - 1).abs().max()) <= 2 * R.unit(dtype) + 40 * R.E32 * lens[0]
    assert bool(got[0][0].isfinite().all())


@pytest.mark.parametrize("new", [1, 12, 60])
@pytest.mark.parametrize("dt,size", [("f16", 9.9e6), ("bf16", 9.9e8), ("f32", 1e30)])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores(dt, size, new, sign):
    """Equal scores of the largest size that is allowed: rows are means of what they see.  Weights are
    rounded once (u), and so is out; sums of n values are off by n 2^-24."""
    dtype, gen, heads, dim, page, n = DTYPES[dt], torch.Generator().manual_seed(35), 2, 64, 16, 150
    v = normal(gen, n, heads, dim, dtype=dtype)
    q, k = torch.full((new, 4, dim), 4.0 * sign, dtype=dtype), torch.full((n, heads, dim), 4.0, dtype=dtype)
    op, pool, table, _, rv = rounded_cache(k, v, [n], page, dtype, gen)
    att = A.mdcn_attention_create(4, heads, dim, True, size / (16 * dim))
    out, lse = K.attend(att, op, q.cuda(), pool, table, ints([n]), ints([0, new]))
    rv = rv.repeat_interleave(2, 1)
    for i in range(new):
        see = rv[:n - new + i + 1]
        bound = R.unit(dtype) * see.mean(0).abs() + (R.unit(dtype) + (n + 16) * R.E32) * see.abs().mean(0)
        within(out[i], (see.mean(0), bound + R.tiny(dtype)), "out")
    seen = torch.arange(n - new + 1, n + 1).double().log()
    within(lse, ((sign * size + seen).expand(4, new), torch.tensor(8 * R.E32 * size)), "lse")
