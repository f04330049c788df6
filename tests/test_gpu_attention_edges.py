"""Attention on the GPU where it can go wrong."""
import math

import pytest
import torch

import attention_reference as R
from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from test_gpu_attention import DTYPES, attend_case, cu, ints, rand, within
from test_gpu_rotary_edges import poison

pytestmark = pytest.mark.gpu
ensure_built()


# ---------------------------------------------------------------- scales

@pytest.mark.parametrize("scale", [1e-44, 1e-38, 3e-38, 1e-30])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_scales_near_zero(dt, scale):
    """Every key has the same weight, and lse is the logarithm of their number."""
    dtype = DTYPES[dt]
    for case in (([70, 3], [130, 5], 4, 2, 64, False), ([1, 2], [2000, 900], 4, 2, 64, True)):
        _, q, k, v, dq, dk, dv, cq, ck = attend_case(case, dtype)
        op = A.mdcn_attention_create(4, 2, 64, case[-1], scale=scale)
        ref = R.attend(q, k, v, cq, ck, None, case[-1], scale, dtype)
        out, lse = A.attend(op, dq, dk, dv, ints(cq), ints(ck))
        within(out, ref["out"], "out")
        within(lse, ref["lse"], "lse")


# ---------------------------------------------------------------- tokens outside every sequence

OUTSIDE = [
    # query tokens, offsets, key tokens, offsets, query heads, key heads
    (300, [10, 200], 260, [0, 50], 2, 1),                    # tile kernel
    (300, [0, 100, 250], 260, [7, 100, 260], 4, 2),
    (5, [1, 2, 4], 9000, [3, 4000, 8000], 4, 2),             # split kernel
    (700, [600, 700], 700, [0, 1], 96, 24),
    (40, [0, 40], 900, [100, 500], 8, 8),                    # parts of dk and dv in the workspace
    (30, [0, 0], 20, [0, 20], 2, 2),
    (6, [0], 7, [0], 2, 2),                                  # no sequences
    (0, [0, 0], 33, [4, 20], 2, 2),                          # no queries
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("case", OUTSIDE, ids=str)
def test_tokens_outside_every_sequence_get_zeros(case, dt, causal):
    """Results that the call allocates are those of a row that sees nothing."""
    tq, cq, tk, ck, hq, hk = case
    dtype = DTYPES[dt]
    op = A.mdcn_attention_create(hq, hk, 64, causal)
    q, k, v = (rand(n, h, 64, seed=s, dtype=dtype) for n, h, s in ((tq, hq, 1), (tk, hk, 2), (tk, hk, 3)))
    go = rand(tq, hq, 64, seed=4, dtype=dtype)
    ref = R.attend(q, k, v, cq, ck, None, causal, op.scale, dtype, go)
    ref = {n: (x[0].masked_fill(x[0].isnan(), -math.inf if n == "lse" else 0.0),
               x[1].masked_fill(x[1].isnan(), 0.0)) for n, x in ref.items()}
    dev = [t.cuda() for t in (q, k, v)]
    go = go.cuda()
    for _ in range(2):
        poison()
        out, lse = A.attend(op, *dev, ints(cq), ints(ck))
        within(out, ref["out"], "out")
        within(lse, ref["lse"], "lse")
        poison()
        g = A.attend_backward(op, *dev, out, lse, go, ints(cq), ints(ck))
        for n in "qkv":
            within(g[n], ref[n], "d" + n)


def test_what_the_caller_gave_is_left_outside_the_sequences():
    op = A.mdcn_attention_create(2, 1, 64, False)
    q = rand(300, 2, 64, seed=1, dtype=torch.float16).cuda()
    for cq, ck in (([10, 200], [0, 50]), ([10, 12], [0, 300])):
        out = torch.full((300, 2, 64), 3.0, dtype=torch.float16, device="cuda")
        lse = torch.full((2, 300), 5.0, device="cuda")
        poison()
        got, own = A.attend(op, q, q[:, :1], q[:, 1:], ints(cq), ints(ck), out=out)
        assert got is out and (out[:10] == 3).all() and (out[cq[1]:] == 3).all()
        assert (own[:, :10] == -math.inf).all() and (own[:, cq[1]:] == -math.inf).all()
        poison()
        own, got = A.attend(op, q, q[:, :1], q[:, 1:], ints(cq), ints(ck), lse=lse)
        assert got is lse and (lse[:, :10] == 5).all() and (lse[:, cq[1]:] == 5).all()
        assert (own[:10] == 0).all() and (own[cq[1]:] == 0).all()


# ---------------------------------------------------------------- fp16 gradients

def half_case(q_scale, k_scale, v_scale, go_scale, keys, seed=0):
    rows, hq, hk, dim = 64, 2, 1, 64
    t = [rand(n, h, dim, seed=seed + i, dtype=torch.float16, scale=s) for i, (n, h, s) in
         enumerate(((rows, hq, q_scale), (keys, hk, k_scale), (keys, hk, v_scale),
                    (rows, hq, go_scale)))]
    op = A.mdcn_attention_create(hq, hk, dim, False)
    want = R.attend(*t[:3], [0, rows], [0, keys], None, False, op.scale, torch.float16, t[3])
    dev = [x.cuda() for x in t]
    c = ints([0, rows]), ints([0, keys])
    out, lse = A.attend(op, *dev[:3], *c)
    return A.attend_backward(op, *dev[:3], out, lse, dev[3], *c), want


def rounding_error(got, exact):
    """The error in units of what rounding the exact values to fp16 leaves."""
    last = (exact.to(torch.float16).double() - exact).norm()
    return float((got.double().cpu() - exact).norm() / last)


@pytest.mark.parametrize("name,scales", [
    # few queries and many keys: p and p (go v - delta) lie far below fp16's normal numbers (6e-5),
    # the gradients within them
    ("q", (2.0 ** -6, 2.0 ** 6, 1.0, 2.0 ** -9)), ("q", (2.0 ** -8, 2.0 ** 8, 1.0, 2.0 ** -13)),
    ("k", (2.0 ** 7, 2.0 ** -7, 1.0, 2.0 ** -4)), ("v", (1.0, 1.0, 1.0, 2.0 ** 5)),
])
def test_half_gradients_of_small_score_gradients(name, scales):
    """As test_score_gradients_carry_two_roundings: two roundings of one size, sqrt(2) = 1.42
    times one alone, and 0.08 for the rounding of out, wherever the factors lie."""
    got, want = half_case(*scales, keys=16384 if name != "v" else 65536)
    assert want[name][0].abs().median() > 2.0 ** -13
    assert rounding_error(got[name], want[name][0]) < 1.5


@pytest.mark.parametrize("name,scales,keys", [
    # go v - delta passes 65504 where the sums' other factor is small
    ("q", (2.0 ** 6, 2.0 ** -6, 2.0 ** 4, 2.0 ** 13), 300),
    ("k", (2.0 ** -7, 2.0 ** 7, 2.0 ** 3, 2.0 ** 13), 300),
    ("q", (2.0 ** 9, 2.0 ** -9, 2.0 ** 8, 2.0 ** 9), 300),
])
def test_half_gradients_of_large_score_gradients(name, scales, keys):
    got, want = half_case(*scales, keys=keys)
    assert want[name][0].abs().max() < 60000
    assert rounding_error(got[name], want[name][0]) < 1.5


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gradients_of_rows_without_gradient_and_of_zeros(dt):
    """All-zero gradients, zero values, single rows that are not zero."""
    dtype = DTYPES[dt]
    op, q, k, v, dq, dk, dv, cq, ck = attend_case(([200, 40], None, 4, 2, 64, True), dtype)
    go = torch.zeros_like(q)
    for rows in ([], [3], [0, 199, 239]):
        for r in rows:
            go[r] = rand(4, 64, seed=r, dtype=dtype)
        ref = R.attend(q, k, v, cq, ck, None, True, op.scale, dtype, go)
        out, lse = A.attend(op, dq, dk, dv, ints(cq), ints(ck))
        g = A.attend_backward(op, dq, dk, dv, out, lse, go.cuda(), ints(cq), ints(ck))
        for n in "qkv":
            within(g[n], ref[n], "d" + n)
        if not rows:
            assert all((g[n] == 0).all() for n in "qkv")


# ---------------------------------------------------------------- small probabilities

@pytest.mark.parametrize("sink", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("heads,rows,n", [(1, 1, 65536), (16, 600, 4096), (32, 1200, 4096)])
@pytest.mark.parametrize("power", [19.3, 21.7, 23.2])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_many_keys_of_little_weight(dt, power, heads, rows, n, sink):
    """One key of weight 1 whose value is 0, and all others of 2^-power with the value 1.  Off by
    the rounding of the weights, scaled by 2^7 in fp16 (half a step 2^-32 below its normal
    numbers), that of the result, and fp32 sums over all keys."""
    dtype = DTYPES[dt]
    op = A.mdcn_attention_create(heads, heads, 8, False, scale=1.0)
    q, k, v = torch.zeros(rows, heads, 8), torch.zeros(n, heads, 8), torch.ones(n, heads, 8)
    q[..., 0] = 1.0
    at = int(sink * (n - 1))
    k[at, :, 0] = power * math.log(2.0)
    v[at] = 0.0
    q, k, v = (t.to(dtype).cuda() for t in (q, k, v))
    out, lse = A.attend(op, q, k, v, ints([0, rows]), ints([0, n]))
    score = float(k[at, 0, 0])
    mass = (n - 1) * math.exp(-score)
    want, least = mass / (1 + mass), 2.0 ** -32 if dtype == torch.float16 else 0.0
    bound = want * (2 * R.unit(dtype) + 2 * n * R.E32) + n * least
    assert float((out.double() - want).abs().max()) <= bound
    assert float((lse.double() - score - math.log1p(mass)).abs().max()) <= n * R.E32


# ---------------------------------------------------------------- layouts

def laid_out(x, how):
    """x [tokens, heads, dim] on the GPU in a layout of its own."""
    n, h, d = x.shape
    pad = 8
    if how == "heads first":
        return x.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    if how == "wide rows":
        w = torch.full((n, h + 3, d + pad), math.nan, dtype=x.dtype, device="cuda")
        v = w[:, 1:h + 1, :d]
    elif how == "interleaved":
        w = torch.full((n, h, 3, d), math.nan, dtype=x.dtype, device="cuda")
        v = w[:, :, 1]
    elif how == "every other token":
        w = torch.full((n, 2, h, d), math.nan, dtype=x.dtype, device="cuda")
        v = w[:, 0]
    else:                                                # heads first, in rows of their own
        w = torch.full((h, n + 2, d + 2 * pad), math.nan, dtype=x.dtype, device="cuda")
        v = w[:, :n, :d].transpose(0, 1)
    v.copy_(x)
    return v


LAYOUTS = ["heads first", "wide rows", "interleaved", "every other token", "heads first, padded"]


@pytest.mark.parametrize("turn", range(5))
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("case", [
    (([150, 3, 40], [170, 60, 40], 4, 2, 96, True), None),
    (([150, 3, 40], [170, 60, 40], 4, 2, 80, False), [170, 33, 0]),
    (([600], [700], 2, 2, 120, True), None),                 # four waves to the keys
    (([130, 65, 1, 100], [130, 75, 1, 100], 96, 24, 40, True), None),
    (([2, 1], [2500, 1300], 8, 2, 96, True), [2500, 1000]),  # split kernel
    (([1, 1], [2500, 1300], 8, 2, 120, True), [2001, 0]),
], ids=str)
def test_layouts(case, dt, turn):
    """Queries, keys, values, outputs and gradients with strides of their own."""
    (ql, kl, hq, hk, dim, causal), used = case
    dtype = DTYPES[dt]
    q, go = (rand(sum(ql), hq, dim, seed=s, dtype=dtype) for s in (1, 2))
    k, v = (rand(sum(kl), hk, dim, seed=s, dtype=dtype) for s in (3, 4))
    op = A.mdcn_attention_create(hq, hk, dim, causal)
    cq, ck = cu(ql), cu(kl)
    ref = R.attend(q, k, v, cq, ck, used, causal, op.scale, dtype, go)
    how = LAYOUTS[turn:] + LAYOUTS[:turn]
    d = [laid_out(x, h) for x, h in zip((q, k, v, torch.zeros_like(q), go), how)]
    more = dict(used_k=None if used is None else ints(used))
    out, lse = A.attend(op, *d[:3], ints(cq), ints(ck), out=d[3], **more)
    assert out is d[3]
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")
    g = A.attend_backward(op, *d[:3], out, lse, d[4], ints(cq), ints(ck), **more)
    for n in "qkv":
        within(g[n], ref[n], "d" + n)
