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
