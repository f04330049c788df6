"""The attention operators on the GPU against their 64-bit reference."""
import math

import pytest
import torch

import attention_reference as R
from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from modulated_deformable_convolution_amd import mdcn

pytestmark = pytest.mark.gpu
ensure_built()

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rand(*shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


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


# ---------------------------------------------------------------- rotary positions

ROTARY = [
    # tokens, q heads, k heads, dim, axes, far, adjacent, round robin, per axis, base
    (1, 1, 1, 2, [1], 0, False, False, False, 10000.0),
    (5, 3, 1, 64, [32], 7, False, False, False, 10000.0),
    (33, 4, 4, 64, [16, 16], 0, True, False, True, 100.0),
    (17, 7, 1, 128, [16, 24, 24], 1000000, False, True, False, 10000.0),
    (3, 16, 4, 80, [14, 13, 13], 2000000000, True, True, False, 10000.0),
    (9, 2, 2, 96, [12, 12, 12], 5, False, False, True, 10000.0),
    (4, 2, 1, 96, [24], -300, False, False, False, 1000000.0),
    (6, 5, 2, 256, [43, 43, 42], 100, False, False, False, 10000.0),
    (2, 2, 1, 250, [63, 62], 3, False, True, False, 10000.0),
    (700, 32, 8, 32, [8], 0, False, False, False, 10000.0),
    (5, 0, 3, 16, [5], 0, False, False, False, 10000.0),
    (5, 3, 0, 16, [3, 0, 2], 0, True, True, True, 10000.0),
]


def rotary_case(case, dtype, sliced, seed=0):
    t, hq, hk, dim, axes, far, adjacent, rr, pa, base = case
    op = A.mdcn_rotary_create(dim, axes, base=base, adjacent=adjacent, round_robin=rr, per_axis=pa)
    x = rand(t, hq + 2 * hk, dim, seed=seed, dtype=dtype)
    q, k = x[:, :hq], x[:, hq:hq + hk]
    if not sliced:
        q, k = q.contiguous(), k.contiguous()
    g = torch.Generator().manual_seed(seed + 1)
    pos = torch.randint(0, 500, (len(axes), t), generator=g) + far
    theta = R.angles(axes, base, rr, pa, pos)
    dev = x.cuda()
    dq, dk = (dev[:, :hq], dev[:, hq:hq + hk]) if sliced else (q.cuda(), k.cuda())
    return op, q, k, dq, dk, pos.to(torch.int32).cuda(), theta, adjacent


@pytest.mark.parametrize("sliced", [False, True])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("case", ROTARY, ids=str)
def test_rotate(case, dt, sliced):
    dtype = DTYPES[dt]
    op, q, k, dq, dk, pos, theta, adj = rotary_case(case, dtype, sliced)
    a, b = A.rotate(op, dq, dk, pos)
    within(a, R.rotate(q, theta, adj, dtype), "q")
    within(b, R.rotate(k, theta, adj, dtype), "k")
    a, b = A.rotate_backward(op, dq, dk, pos)
    within(a, R.rotate(q, -theta, adj, dtype), "q back")
    within(b, R.rotate(k, -theta, adj, dtype), "k back")
    A.rotate(op, dq, dk, pos, q_out=dq, k_out=dk)
    within(dq, R.rotate(q, theta, adj, dtype), "q in place")
    within(dk, R.rotate(k, theta, adj, dtype), "k in place")


@pytest.mark.parametrize("sliced", [False, True])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("case", ROTARY, ids=str)
def test_norm_rotate(case, dt, sliced):
    dtype = DTYPES[dt]
    op, q, k, dq, dk, pos, theta, adj = rotary_case(case, dtype, sliced, seed=3)
    dim = q.shape[-1]
    wq, wk = (rand(dim, seed=s, dtype=torch.float32, scale=0.2).add(1).to(dtype) for s in (5, 6))
    eps = 1e-6
    a, b = A.norm_rotate(op, dq, dk, pos, wq.cuda(), wk.cuda(), eps)
    within(a, R.norm_rotate(q, wq, eps, theta, adj, dtype), "q")
    within(b, R.norm_rotate(k, wk, eps, theta, adj, dtype), "k")
    gq, gk = rand(*q.shape, seed=7, dtype=dtype), rand(*k.shape, seed=8, dtype=dtype)
    g = A.norm_rotate_backward(op, dq, dk, pos, wq.cuda(), wk.cuda(), gq.cuda(), gk.cuda(), eps)
    for n, x, w, gy in (("q", q, wq, gq), ("k", k, wk, gk)):
        dx, dw = R.norm_rotate_backward(x, w, eps, theta, adj, gy, dtype)
        within(g[n], dx, "d" + n)
        if x.shape[1]:
            within(g[n + "_gain"], dw, "d gain of " + n)


def test_norm_rotate_zero_rows_and_no_tokens():
    op = A.mdcn_rotary_create(64, [16, 16])
    x = torch.zeros(4, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    pos = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    a, b = A.norm_rotate(op, x, x[:, :1], pos, w, w)
    assert (a == 0).all() and (b == 0).all()
    e = x[:0]
    g = A.norm_rotate_backward(op, e, e, pos[:, :0], w, w, e, e)
    assert (g["q_gain"] == 0).all() and (g["k_gain"] == 0).all() and g["q"].shape == (0, 2, 64)
    a, b = A.rotate(op, e, e, pos[:, :0])
    assert a.shape == (0, 2, 64)


def test_gain_gradients_repeat_to_the_bit():
    op = A.mdcn_rotary_create(64, [32])
    q = rand(5000, 4, 64, seed=1, dtype=torch.float32).cuda()
    w = torch.ones(64, device="cuda")
    pos = torch.arange(5000, dtype=torch.int32, device="cuda")[None]
    runs = [A.norm_rotate_backward(op, q, q, pos, w, w, q, q) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(r[n], runs[0][n]) for n in r)


# ---------------------------------------------------------------- attention

ATTEND = [
    # q lens, k lens (None: the same), q heads, k heads, dim, causal
    ([1], None, 1, 1, 8, True),
    ([1, 0, 2, 31, 32, 33], None, 4, 2, 64, True),
    ([63, 64, 65, 0, 1], None, 2, 1, 128, True),
    ([127, 130, 1], None, 3, 3, 32, False),
    ([200, 129], None, 4, 4, 80, True),
    ([70, 3, 0, 50], [30, 200, 5, 0], 8, 2, 96, True),       # rows that see nothing, no keys, no queries
    ([70, 3, 0, 50], [30, 200, 5, 0], 8, 2, 96, False),
    ([5, 150], [300, 161], 7, 1, 128, True),
    ([40, 100], [290, 33], 6, 2, 40, False),
    ([260], [700], 2, 2, 24, True),
]


def attend_case(case, dtype, seed=0, sliced=True):
    ql, kl, hq, hk, dim, causal = case
    kl = kl or ql
    op = A.mdcn_attention_create(hq, hk, dim, causal)
    q = rand(sum(ql), hq, dim, seed=seed, dtype=dtype)
    kv = rand(sum(kl), 2 * hk, dim, seed=seed + 1, dtype=dtype)
    k, v = kv[:, :hk], kv[:, hk:]
    dev = kv.cuda()
    dk, dv = (dev[:, :hk], dev[:, hk:]) if sliced else (k.contiguous().cuda(), v.contiguous().cuda())
    return op, q, k, v, q.cuda(), dk, dv, cu(ql), cu(kl)


def check_attend(case, dtype, train=True, used=None, seed=0):
    op, q, k, v, dq, dk, dv, cq, ck = attend_case(case, dtype, seed)
    go = rand(*q.shape, seed=seed + 9, dtype=dtype)
    ref = R.attend(q, k, v, cq, ck, used, op.causal, op.scale, dtype, go if train else None)
    dused = None if used is None else ints(used)
    out, lse = A.attend(op, dq, dk, dv, ints(cq), ints(ck), used_k=dused)
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")
    if train:
        g = A.attend_backward(op, dq, dk, dv, out, lse, go.cuda(), ints(cq), ints(ck), used_k=dused)
        for n in "qkv":
            within(g[n], ref[n], "d" + n)
    return out, lse


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("case", ATTEND, ids=str)
def test_attend(case, dt):
    check_attend(case, DTYPES[dt])


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("dim", [8, 16, 48, 56, 64, 72, 104, 120, 128])
def test_attend_dims(dim, dt):
    check_attend(([37, 130], None, 2, 1, dim, True), DTYPES[dt])
    check_attend(([2, 1], [37, 130], 2, 1, dim, True), DTYPES[dt])
    check_attend(([2, 1], [2500, 1300], 2, 1, dim, True), DTYPES[dt], train=False)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("new", [1, 2, 5])
@pytest.mark.parametrize("heads", [(8, 2), (7, 1), (4, 4), (32, 1)])
@pytest.mark.parametrize("size", [300, 2600])
def test_decode(size, heads, new, dt):
    hq, hk = heads
    used = [new, size, 31, 32, 33, 0, 257, 64, 128, 1, size - 1]
    case = ([new] * len(used), [size] * len(used), hq, hk, 64 if new == 2 else 128, True)
    check_attend(case, DTYPES[dt], train=False, used=used)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_decode_long(dt):
    # several workgroups share a sequence, and one takes several sequences
    for batch, lens in ((1, [20000]), (3, [9000, 17, 12001]), (130, None)):
        lens = lens or [(i * 37) % 150 for i in range(batch)]
        case = ([1] * batch, [max(lens)] * batch, 2, 1, 128, True)
        check_attend(case, DTYPES[dt], train=False, used=lens)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_training_against_a_partly_used_cache(dt):
    check_attend(([40, 3, 70], [100, 60, 90], 4, 2, 64, True), DTYPES[dt], used=[77, 0, 90])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("rows,size", [(1, 250), (3, 250), (200, 250), (1, 3001), (3, 3001)])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_unused_cache_rows_are_never_used(dt, rows, size, causal):
    dtype = DTYPES[dt]
    case = ([rows, rows], [size, 333], 4, 2, 64, causal)
    op, q, k, v, dq, dk, dv, cq, ck = attend_case(case, dtype)
    used = [211, 33]
    for x in (dk, dv):
        for b in range(2):
            x[ck[b] + used[b]:ck[b + 1]] = math.nan
    ref = R.attend(q, k, v, cq, ck, used, causal, op.scale, dtype)
    out, lse = A.attend(op, dq, dk, dv, ints(cq), ints(ck), used_k=ints(used))
    within(out, ref["out"], "out")
    within(lse, ref["lse"], "lse")


LONG = [
    # few heads of long sequences: workgroups no more than the compute units
    ([700], None, 2, 1, 64, True),
    ([515], None, 2, 2, 128, False),
    ([130, 700, 1], [1100, 700, 300], 3, 1, 32, True),
    ([90, 400], [1300, 33], 2, 1, 80, True),               # rows that see nothing
    ([700], [1025], 2, 1, 96, False),
]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_sequences_of_few_heads(case, dt):
    check_attend(case, DTYPES[dt])


@pytest.mark.parametrize("at", [1023, 1000, 700, 100])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_hidden_rows_of_long_sequences(dt, at):
    """As the two tests below, where waves share a row's keys."""
    dtype = DTYPES[dt]
    op, q, k, v, dq, dk, dv, cq, ck = attend_case(([1024], None, 2, 1, 128, True), dtype)
    go = rand(*q.shape, seed=9, dtype=dtype)
    ref = R.attend(q, k, v, cq, ck, None, True, op.scale, dtype, go)
    for x in (dv, dk):
        x[at] = math.nan
        out, lse = A.attend(op, dq, dk, dv, ints(cq), ints(ck))
        got = A.attend_backward(op, dq, dk, dv, out, lse, go.cuda(), ints(cq), ints(ck))["q"]
        within(out[:at], (ref["out"][0][:at], ref["out"][1][:at]), "out")
        within(got[:at], (ref["q"][0][:at], ref["q"][1][:at]), "dq")
        assert not out[at:].isfinite().any() and not got[at:].isfinite().all(-1).any()


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("rows,keys", [(4, 170), (150, 170), (4, 3000)])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_hidden_values_reach_no_row(dt, rows, keys, value):
    """A row of k and v that is not finite shows in the rows that see it only."""
    dtype = DTYPES[dt]
    case = ([rows, 3], [keys, 3], 2, 1, 64, True)
    op, q, k, v, dq, dk, dv, cq, ck = attend_case(case, dtype)
    at = keys - 2                                       # seen by the last two rows of sequence 0
    ref = R.attend(q, k, v, cq, ck, None, True, op.scale, dtype)
    for x in (dv, dk):
        x[at] = value
        out, lse = A.attend(op, dq, dk, dv, ints(cq), ints(ck))
        out = out.double().cpu()
        clean = torch.ones(q.shape[0], dtype=torch.bool)
        clean[rows - 2:rows] = False
        within(out[clean], (ref["out"][0][clean], ref["out"][1][clean]), "rows that do not see it")
        assert not out[~clean].isfinite().any()


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_hidden_keys_reach_no_query_gradient(dt, value):
    dtype = DTYPES[dt]
    case = ([150, 3], [170, 3], 2, 1, 64, True)
    op, q, k, v, dq, dk, dv, cq, ck = attend_case(case, dtype)
    go = rand(*q.shape, seed=9, dtype=dtype)
    ref = R.attend(q, k, v, cq, ck, None, True, op.scale, dtype, go)
    clean = torch.ones(153, dtype=torch.bool)
    clean[148:150] = False                             # the rows that see key 168
    for x in (dv, dk):
        x[168] = value
        out, lse = A.attend(op, dq, dk, dv, ints(cq), ints(ck))
        got = A.attend_backward(op, dq, dk, dv, out, lse, go.cuda(), ints(cq), ints(ck))["q"]
        within(got[clean.cuda()], (ref["q"][0][clean], ref["q"][1][clean]), "dq")
        assert not got[~clean.cuda()].isfinite().all(-1).any()


def test_masked_rows_with_extreme_scores():
    """Scores at the ends of the range: the softmax stays exact where it is defined."""
    for dtype in DTYPES.values():
        op = A.mdcn_attention_create(1, 1, 8, False)
        q = torch.zeros(200, 1, 8, dtype=dtype)
        k, v = torch.zeros(90, 1, 8, dtype=dtype), rand(90, 1, 8, seed=1, dtype=dtype)
        q[:, 0, 0] = 200.0
        k[:, 0, 0] = torch.linspace(-200, 200, 90).to(dtype)
        out, lse = A.attend(op, q.cuda(), k.cuda(), v.cuda(), ints([0, 200]), ints([0, 90]))
        ref = R.attend(q, k, v, [0, 200], [0, 90], None, False, op.scale, dtype)
        within(out, ref["out"], "out")
        within(lse, ref["lse"], "lse")


@pytest.mark.parametrize("dim", [32, 80, 128])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_a_row_that_sees_one_key_has_no_score_gradient(dt, dim):
    """softmax of one score is 1 whatever the score: dq and dk are exactly zero."""
    dtype = DTYPES[dt]
    n = 70
    op = A.mdcn_attention_create(4, 2, dim, True)
    q, k, v, go = (rand(n, h, dim, seed=s, dtype=dtype).cuda()
                   for s, h in ((1, 4), (2, 2), (3, 2), (4, 4)))
    c = ints(list(range(n + 1)))
    out, lse = A.attend(op, q, k, v, c, c)
    g = A.attend_backward(op, q, k, v, out, lse, go, c, c)
    assert torch.equal(out, v.repeat_interleave(2, 1))
    assert (g["q"] == 0).all() and (g["k"] == 0).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[2] * 40, [8] * 20, [33, 70, 5, 1, 31], [300]], ids=str)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_score_gradients_carry_two_roundings(dt, lens, causal):
    """dq and dk: the score gradients are rounded for the product and the results once more, which
    are errors of one size and independent, sqrt(2) = 1.42 times the last one's alone.  The
    rounding of out, which is an input here, adds less than 0.08 of them in rows of
    more than 32 keys, and nothing in rows of fewer."""
    dtype = DTYPES[dt]
    n, c = sum(lens), cu(lens)
    q, k, v, go = (rand(n, 8, 64, seed=60 + i, dtype=dtype) for i in range(4))
    op = A.mdcn_attention_create(8, 8, 64, causal)
    dev = [t.cuda() for t in (q, k, v)]
    out, lse = A.attend(op, *dev, ints(c), ints(c))
    got = A.attend_backward(op, *dev, out, lse, go.cuda(), ints(c), ints(c))
    want = R.attend(q, k, v, c, c, None, causal, 64 ** -0.5, dtype, go)
    for name in ("q", "k"):
        exact = want[name][0]
        last = (exact.to(dtype).double() - exact).norm()
        assert float((got[name].double().cpu() - exact).norm() / last) < 1.5, name


def test_gradients_repeat_to_the_bit_and_match_differences():
    case = ([50, 90], None, 4, 2, 32, True)
    op, q, k, v, dq, dk, dv, cq, ck = attend_case(case, torch.float32)
    go = rand(*q.shape, seed=4, dtype=torch.float32)
    out, lse = A.attend(op, dq, dk, dv, ints(cq), ints(ck))
    runs = [A.attend_backward(op, dq, dk, dv, out, lse, go.cuda(), ints(cq), ints(ck))
            for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(r[n], runs[0][n]) for n in r)
    ref = R.attend(q, k, v, cq, ck, None, True, op.scale, torch.float32, go)

    def loss(q, k, v):
        return float((R.attend(q, k, v, cq, ck, None, True, op.scale,
                               torch.float32)["out"][0] * go.double()).sum())
    x = {"q": q.double(), "k": k.double(), "v": v.double()}
    for n in "qkv":
        d = torch.randn(x[n].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(5))
        h = 1e-5
        diff = (loss(**{**x, n: x[n] + h * d}) - loss(**{**x, n: x[n] - h * d})) / (2 * h)
        got = float((runs[0][n].double().cpu() * d).sum())
        assert abs(got - diff) <= float((ref[n][1] * d.abs()).sum()) + 1e-6


def test_attend_far_into_a_cache():
    """Rows past 2^32 bytes of a cache."""
    size, hk, dim = 280000, 64, 128
    op = A.mdcn_attention_create(hk, hk, dim, True)
    k = torch.empty((size, hk, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    start = size - 600
    k[start:] = rand(600, hk, dim, seed=1, dtype=torch.bfloat16).cuda()
    v[start:] = rand(600, hk, dim, seed=2, dtype=torch.bfloat16).cuda()
    for rows in (1, 130):
        q = rand(rows, hk, dim, seed=3, dtype=torch.bfloat16)
        out, lse = A.attend(op, q.cuda(), k, v, ints([0, 0, rows]), ints([0, start, size]))
        ref = R.attend(q, k[start:].cpu(), v[start:].cpu(), [0, rows], [0, 600], None, True,
                       op.scale, torch.bfloat16)
        within(out, ref["out"], "out")
        within(lse, ref["lse"], "lse")


def test_offsets_outside_the_tensors_stay_inside():
    op = A.mdcn_attention_create(2, 1, 64, True)
    q, kv = rand(20, 2, 64, seed=1, dtype=torch.bfloat16).cuda(), \
        rand(20, 1, 64, seed=2, dtype=torch.bfloat16).cuda()
    cache = torch.zeros(7000, 1, 64, dtype=torch.bfloat16, device="cuda")
    for offsets in ([0, 1 << 30], [-5, 400, 20], [20, 3, -7], [7, 7, 7], [1 << 30, -(1 << 30)]):
        out = torch.full((20, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        out, lse = A.attend(op, q, kv, kv, ints(offsets), ints(offsets), out=out)
        A.attend_backward(op, q, kv, kv, out, lse, q, ints(offsets), ints(offsets))
        used = ints([1 << 30] * (len(offsets) - 1))
        A.attend(op, q[:2], kv, kv, ints(offsets), ints(offsets), used_k=used)
        A.attend(op, q[:2], cache, cache, ints(offsets), ints([min(5000 * v, 1 << 30) for v in offsets[:-1]] +
                                                              [7000]), used_k=used)
    # sequences that all claim the whole cache
    many = ints([0, 2] * 300 + [0])
    A.attend(op, q[:2], cache, cache, many, ints([0, 7000] * 300 + [0]))
    torch.cuda.synchronize()


def test_tokens_outside_every_sequence_are_left():
    op = A.mdcn_attention_create(2, 1, 64, False)
    q = rand(300, 2, 64, seed=1, dtype=torch.float16).cuda()
    out = torch.full((300, 2, 64), 3.0, dtype=torch.float16, device="cuda")
    A.attend(op, q, q[:, :1], q[:, 1:], ints([10, 200]), ints([0, 50]), out=out)
    assert (out[:10] == 3).all() and (out[200:] == 3).all() and not (out[10:200] == 3).any()


def test_other_stream_and_graph():
    """On a stream of its own, and captured: every replay equals the eager result."""
    op = A.mdcn_attention_create(4, 2, 64, True)
    rot = A.mdcn_rotary_create(64, [16, 16])
    case = ([30, 200], None, 4, 2, 64, True)
    _, _, _, _, q, k, v, cq, ck = attend_case(case, torch.bfloat16)
    cq, ck = ints(cq), ints(ck)
    pos = torch.arange(460, dtype=torch.int32, device="cuda").view(2, 230)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    go = rand(230, 4, 64, seed=3, dtype=torch.bfloat16).cuda()

    def step():
        a, b = A.norm_rotate(rot, q, k, pos, w, w)
        out, lse = A.attend(op, a, b, v, cq, ck)
        g = A.attend_backward(op, a, b, v, out, lse, go, cq, ck)
        n = A.norm_rotate_backward(rot, q, k, pos, w, w, g["q"], g["k"])
        d, _ = A.attend(op, a[:2], b, v, ints_cu, ck)
        return [out, lse, d, g["v"]] + [n[i] for i in sorted(n)]

    ints_cu = ints([0, 1, 2])
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out, _ = A.attend(op, q, k, v, cq, ck, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, A.attend(op, q, k, v, cq, ck)[0])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        assert all(torch.equal(a, b) for a, b in zip(step(), want)), i


def test_bad_tensors_are_refused():
    op = A.mdcn_attention_create(4, 2, 64, True)
    q = torch.zeros(10, 4, 64, device="cuda")
    k = torch.zeros(10, 2, 64, device="cuda")
    c = ints([0, 10])
    bad = [
        (q[:, :3], k, k, c, c), (q, k[:, :1], k, c, c), (q, k, k[:9], c, c),
        (q[:, :, :32], k, k, c, c), (q.half(), k, k, c, c), (q, k, k, c.long(), c),
        (q, k, k, c, ints([0, 5, 10])), (q, k.transpose(0, 1).contiguous(), k, c, c),
        (torch.zeros(10, 64, 4, device="cuda").transpose(1, 2), k, k, c, c),
        (torch.zeros(10, 4, 65, device="cuda")[:, :, 1:], k, k, c, c), (q.double(), k, k, c, c),
        (torch.zeros(10, 4, 64, dtype=torch.int32, device="cuda"), k, k, c, c),
    ]
    for args in bad:
        with pytest.raises(mdcn.MdcnError):
            A.attend(op, *args)
    with pytest.raises(mdcn.MdcnError):
        A.attend(op, q, k, k, c, c, used_k=ints([1, 2]))
    with pytest.raises(mdcn.MdcnError):
        A.attend(op, q, k, k, c, c, out=q)
    with pytest.raises(mdcn.MdcnError):
        A.attend(op, q, k, k, c, c, lse=torch.zeros(10, 4, device="cuda"))
    rot = A.mdcn_rotary_create(64, [16, 16])
    pos = torch.zeros(2, 10, dtype=torch.int32, device="cuda")
    for args in ((q, k, pos[:1]), (q, k, pos.long()), (q, k[:9], pos), (q, k.half(), pos),
                 (q[..., :32], k, pos)):
        with pytest.raises(mdcn.MdcnError):
            A.rotate(rot, *args)
    w = torch.ones(64, device="cuda")
    with pytest.raises(mdcn.MdcnError):
        A.norm_rotate(rot, q, k, pos, w[:32], w)
    with pytest.raises(mdcn.MdcnError):
        A.norm_rotate(rot, q, k, pos, w.half(), w)
