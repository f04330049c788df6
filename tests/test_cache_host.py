"""Host checks of the cache and page entry points: what they refuse, before any GPU is
asked for anything (the pointers here are addresses that nothing reads)."""
import ctypes

import pytest
import torch

import cache_reference as C
from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from modulated_deformable_convolution_amd import cache as K
from modulated_deformable_convolution_amd import mdcn

ensure_built()
BASE = 1 << 30
STEP = 1 << 24


def at(i):
    return BASE + i * STEP


def dims(v):
    return (ctypes.c_int64 * len(v))(*v)


def status(name):
    return getattr(mdcn, "MDCN_E_" + name)


# ---------------------------------------------------------------- handles

@pytest.mark.parametrize("kw", [
    dict(k_heads=0), dict(k_heads=65537), dict(dim=0), dict(dim=12), dict(dim=136), dict(page=0),
    dict(page=8), dict(page=24), dict(page=512), dict(page=-16),
])
def test_create_refuses(kw):
    with pytest.raises(mdcn.MdcnError) as e:
        K.mdcn_cache_create(**{**dict(k_heads=2, dim=64, page=16), **kw})
    assert e.value.status == mdcn.MDCN_E_ATTR
    lib = mdcn.library()
    assert lib.mdcn_cache_create(2, 64, 16, None) == mdcn.MDCN_E_NULL
    assert lib.mdcn_cache_page_bytes(None, None) == mdcn.MDCN_E_NULL
    lib.mdcn_cache_destroy(None)


@pytest.mark.parametrize("heads,dim,page", [(1, 8, 16), (3, 40, 32), (8, 96, 64), (8, 128, 256), (2, 64, 128)])
def test_page_bytes(heads, dim, page):
    assert K.mdcn_cache_create(heads, dim, page).page_bytes == C.page_bytes(heads, dim, page)


# ---------------------------------------------------------------- store and load

# batch, tokens, pages, page stride, width, row stride, strides of k and v (2 heads of 64, bf16)
GOOD = [3, 10, 20, 4 * 1088, 5, 6, 256, 64, 256, 64]


def moved(op, d, load=False, dtype=2, k=at(0), v=at(1), table=at(2), used=at(3), cu=at(4), pool=at(5)):
    lib = mdcn.library()
    if load:
        return lib.mdcn_cache_load(op, dtype, d, pool, table, used, cu, 0, k, v, None)
    return lib.mdcn_cache_store(op, dtype, d, k, v, table, used, cu, pool, None)


@pytest.fixture(scope="module")
def cache():
    return K.mdcn_cache_create(2, 64, 32)


@pytest.mark.parametrize("load", [False, True])
@pytest.mark.parametrize("change,code", [
    ({0: -1}, "SHAPE"), ({0: 1 << 25}, "SHAPE"), ({1: -1}, "SHAPE"), ({1: 1 << 31}, "SHAPE"),
    ({2: -1}, "SHAPE"), ({2: 1 << 31}, "SHAPE"), ({3: 4 * 1088 - 16}, "SHAPE"), ({3: 4 * 1088 + 8}, "SHAPE"),
    ({3: -16}, "SHAPE"), ({3: 1 << 32}, "SHAPE"), ({4: -1}, "SHAPE"), ({4: 1 << 26}, "SHAPE"),
    ({5: 4}, "SHAPE"), ({6: 60}, "SHAPE"), ({6: 260}, "SHAPE"), ({7: 4}, "SHAPE"), ({8: -256}, "SHAPE"),
    ({9: 1 << 41}, "SHAPE"),
])
def test_moves_refuse_dims(cache, change, code, load):
    d = list(GOOD)
    for i, v in change.items():
        d[i] = v
    assert moved(cache.handle, dims(d), load) == status(code)


@pytest.mark.parametrize("load", [False, True])
def test_moves_refuse_pointers(cache, load):
    d = dims(GOOD)
    for n in ("k", "v", "table", "used", "cu", "pool"):
        assert moved(cache.handle, d, load, **{n: None}) == mdcn.MDCN_E_NULL
    assert moved(None, d, load) == mdcn.MDCN_E_NULL
    assert moved(cache.handle, None, load) == mdcn.MDCN_E_NULL
    assert moved(cache.handle, d, load, dtype=3) == mdcn.MDCN_E_DTYPE
    assert moved(cache.handle, d, load, pool=at(5) + 8) == mdcn.MDCN_E_SHAPE
    assert moved(cache.handle, d, load, k=at(0) + 8) == mdcn.MDCN_E_SHAPE
    for kw in (dict(k=at(5)), dict(v=at(5) + 19 * 4352 + 4336), dict(k=at(5) - 16), dict(table=at(5)),
               dict(used=at(5)), dict(cu=at(5) + 16)):
        assert moved(cache.handle, d, load, **kw) == (mdcn.MDCN_E_ALIAS if not load or kw.keys() & {"k", "v"}
                                                      else mdcn.MDCN_E_DEVICE)
    if load:
        for kw in (dict(k=at(1)), dict(k=at(2)), dict(v=at(3)), dict(k=at(4))):
            assert moved(cache.handle, d, True, **kw) == mdcn.MDCN_E_ALIAS
        assert moved(cache.handle, dims(GOOD[:6] + [256, 32] + GOOD[8:]), True) == mdcn.MDCN_E_ALIAS


def test_nothing_to_move(cache):
    none = list(GOOD)
    none[1] = 0
    assert moved(cache.handle, dims(none), k=None, v=None) == mdcn.MDCN_OK
    none = list(GOOD)
    none[0] = 0
    assert moved(cache.handle, dims(none), table=None, used=None) == mdcn.MDCN_OK
    assert moved(cache.handle, dims(none), True) == mdcn.MDCN_OK


# ---------------------------------------------------------------- attention

# batch, query tokens, pages, page stride, width, row stride, strides of q and out (4 heads of 64)
GOOD_ATT = [3, 10, 20, 4 * 1088, 5, 6, 256, 64, 256, 64]


def attended(att, op, d, dtype=2, q=at(0), pool=at(1), table=at(2), used=at(3), cu=at(4), out=at(6),
             lse=at(7), ws=at(8), ws_bytes=STEP):
    return mdcn.library().mdcn_cache_attend(att, op, dtype, d, q, pool, table, used, cu, 0, out, lse, ws,
                                            ws_bytes, None)


def need(att, op, d, dtype=2):
    n = ctypes.c_size_t()
    assert mdcn.library().mdcn_cache_attend_workspace_bytes(att, op, dtype, d, ctypes.byref(n)) == 0
    return n.value


def test_attend_refuses(cache):
    att = A.mdcn_attention_create(4, 2, 64, True)
    d, op = dims(GOOD_ATT), cache.handle
    n = need(att.handle, op, d)
    assert 0 < n <= STEP
    assert attended(att.handle, op, d, ws_bytes=n - 1) == mdcn.MDCN_E_WORKSPACE
    assert attended(att.handle, op, d, ws=None) == mdcn.MDCN_E_WORKSPACE
    for name in ("q", "pool", "table", "used", "cu", "out", "lse"):
        assert attended(att.handle, op, d, **{name: None}) == mdcn.MDCN_E_NULL
    assert attended(None, op, d) == attended(att.handle, None, d) == mdcn.MDCN_E_NULL
    assert attended(att.handle, op, d, dtype=-1) == mdcn.MDCN_E_DTYPE
    for kw in (dict(out=at(0)), dict(out=at(1)), dict(out=at(2)), dict(out=at(7)), dict(lse=at(0)),
               dict(lse=at(1)), dict(ws=at(0)), dict(ws=at(1)), dict(ws=at(4)), dict(ws=at(6)), dict(ws=at(7))):
        assert attended(att.handle, op, d, **kw) == mdcn.MDCN_E_ALIAS
    for change in ({6: 250}, {7: 60}, {8: 128}, {9: 20}, {2: -1}, {4: 1 << 26}):
        bad = list(GOOD_ATT)
        for i, v in change.items():
            bad[i] = v
        assert attended(att.handle, op, dims(bad)) in (mdcn.MDCN_E_SHAPE, mdcn.MDCN_E_ALIAS)
    other = A.mdcn_attention_create(4, 4, 64, True)
    assert attended(other.handle, op, d) == mdcn.MDCN_E_ATTR
    other = A.mdcn_attention_create(4, 2, 32, True)
    assert attended(other.handle, op, d) == mdcn.MDCN_E_ATTR
    assert attended(att.handle, op, d) == mdcn.MDCN_E_DEVICE
    many = A.mdcn_attention_create(8192, 2, 64, True)
    rows = list(GOOD_ATT)
    rows[1] = 1 << 20
    assert attended(many.handle, op, dims(rows)) == mdcn.MDCN_E_SHAPE       # 2^32 rows of a key head


def test_attend_describes(cache):
    att = A.mdcn_attention_create(4, 2, 64, True)
    assert K.describe_attend(att, cache, torch.bfloat16, 48, 48, 1000) == \
        "split rows=16 workgroups=1024 unit=32"
    assert K.describe_attend(att, cache, torch.float16, 48, 48 * 16, 1000) == \
        "split rows=32 workgroups=512 unit=32"
    assert K.describe_attend(att, cache, torch.float16, 2, 2000, 1000) == \
        "tile rows=128 workgroups=512 unit=64"
    assert K.describe_attend(att, cache, torch.float32, 2, 2000, 1000) == \
        "tile rows=64 workgroups=512 unit=64"
    small = K.describe_attend(att, cache, torch.float32, 1, 1, 1)
    assert small.startswith("split rows=16 workgroups=") and int(small.split("=")[2].split()[0]) < 20
    wide = K.describe_attend(att, cache, torch.float16, 4096, 4096, 1 << 24)
    assert int(wide.split("=")[-1]) > 32
    assert mdcn.library().mdcn_describe_cache_attend(att.handle, cache.handle, 2, dims(GOOD_ATT), None, 5) == \
        mdcn.MDCN_E_NULL


# ---------------------------------------------------------------- pages

# layers, pages, bytes, page stride, layer stride, page, rows, rows of the result, width
GOOD_FORK = [2, 30, 544, 544, 30 * 544, 16, 4, 6, 5]


def forked(d, pool=at(0), table=at(1), used=at(2), owners=at(3), parents=at(4), new=at(5), out=(6, 7, 8, 9),
           ws=at(10), ws_bytes=STEP):
    out = [None if i is None else i if i > 1000 else at(i) for i in out]
    return mdcn.library().mdcn_pages_fork(d, pool, table, used, owners, parents, new, *out, ws, ws_bytes, None)


@pytest.mark.parametrize("change", [
    {0: -1}, {1: -1}, {1: 1 << 31}, {2: 540}, {2: -16}, {2: 1 << 31}, {3: 528}, {3: 552}, {4: 8}, {4: 512},
    {4: 29 * 544}, {5: 0}, {5: -1}, {5: (1 << 20) + 1}, {6: -1}, {7: -1}, {8: -1}, {8: 1 << 27},
    {6: 1 << 30}, {7: 1 << 30},
])
def test_fork_refuses_dims(change):
    d = list(GOOD_FORK)
    for i, v in change.items():
        d[i] = v
    assert forked(dims(d)) == mdcn.MDCN_E_SHAPE


def test_fork_refuses_pointers():
    d = dims(GOOD_FORK)
    for kw in (dict(pool=None), dict(table=None), dict(used=None), dict(owners=None), dict(out=(None, 7, 8, 9)),
               dict(out=(6, None, 8, 9)), dict(out=(6, 7, None, 9)), dict(out=(6, 7, 8, None))):
        assert forked(d, **kw) == mdcn.MDCN_E_NULL
    assert forked(None) == mdcn.MDCN_E_NULL
    assert forked(d, parents=None) == mdcn.MDCN_E_SHAPE
    n = ctypes.c_size_t()
    assert mdcn.library().mdcn_pages_fork_workspace_bytes(d, ctypes.byref(n)) == mdcn.MDCN_OK
    assert forked(d, ws_bytes=n.value - 1) == forked(d, ws=None) == mdcn.MDCN_E_WORKSPACE
    for kw in (dict(out=(1, 7, 8, 9)), dict(out=(6, 2, 8, 9)), dict(out=(6, 7, 3, 9)), dict(out=(6, 7, 8, 4)),
               dict(out=(5, 7, 8, 9)), dict(out=(6, 6, 8, 9)), dict(out=(0, 7, 8, 9)), dict(ws=at(1)),
               dict(ws=at(8)), dict(ws=at(0)), dict(table=at(0)),
               dict(out=(6, 7, 8, at(0) + 59 * 544 + 540))):
        assert forked(d, **kw) == mdcn.MDCN_E_ALIAS
    assert forked(d, pool=at(0) + 8) == mdcn.MDCN_E_SHAPE
    assert forked(d) == forked(d, new=None) == mdcn.MDCN_E_DEVICE
    # pages within which the layers lie
    assert forked(dims([2, 30, 544, 1088, 544] + GOOD_FORK[5:])) == mdcn.MDCN_E_DEVICE


def test_compact_refuses():
    def call(d, pool=at(0), table=at(1), owners=at(2), out=(3, 4, 5), ws=at(6), ws_bytes=STEP):
        out = [None if i is None else at(i) for i in out]
        return mdcn.library().mdcn_pages_compact(d, pool, table, owners, *out, ws, ws_bytes, None)

    d = dims(GOOD_FORK[:5] + [4, 5])
    for kw in (dict(pool=None), dict(table=None), dict(owners=None), dict(out=(None, 4, 5)),
               dict(out=(3, None, 5)), dict(out=(3, 4, None))):
        assert call(d, **kw) == mdcn.MDCN_E_NULL
    assert call(None) == mdcn.MDCN_E_NULL
    n = ctypes.c_size_t()
    assert mdcn.library().mdcn_pages_compact_workspace_bytes(d, ctypes.byref(n)) == mdcn.MDCN_OK
    assert call(d, ws_bytes=n.value - 1) == call(d, ws=None) == mdcn.MDCN_E_WORKSPACE
    for kw in (dict(out=(1, 4, 5)), dict(out=(3, 2, 5)), dict(out=(3, 4, 4)), dict(out=(3, 4, 0)),
               dict(ws=at(1)), dict(ws=at(5))):
        assert call(d, **kw) == mdcn.MDCN_E_ALIAS
    for change in ({5: -1}, {6: -1}, {1: -1}, {2: 8}, {6: 1 << 31}):
        bad = GOOD_FORK[:5] + [4, 5]
        for i, v in change.items():
            bad[i] = v
        assert call(dims(bad)) == mdcn.MDCN_E_SHAPE
    assert call(dims([0] * 7), None, None, None, (None, None, None)) == mdcn.MDCN_OK
    assert call(d) == mdcn.MDCN_E_DEVICE


def test_copy_refuses():
    def call(d, src=at(0), dst=at(1), a=at(2), b=at(3)):
        return mdcn.library().mdcn_pages_copy(d, src, dst, a, b, None)

    good = [2, 7, 544, 30, 544, 30 * 544, 20, 544, 20 * 544]
    for kw in (dict(src=None), dict(dst=None), dict(a=None), dict(b=None)):
        assert call(dims(good), **kw) == mdcn.MDCN_E_NULL
    assert call(None) == mdcn.MDCN_E_NULL
    for i, v in ((0, -1), (1, -1), (1, 1 << 31), (2, 536), (3, -1), (4, 540), (5, 29 * 544), (6, 1 << 31),
                 (7, 528), (8, 100)):
        bad = list(good)
        bad[i] = v
        assert call(dims(bad)) == mdcn.MDCN_E_SHAPE
    assert call(dims(good), a=at(1)) == call(dims(good), b=at(1) + 544) == mdcn.MDCN_E_ALIAS
    assert call(dims(good), dst=at(0)) == mdcn.MDCN_E_ALIAS                  # one address, other strides
    same = good[:6] + good[3:6]
    assert call(dims(same), dst=at(0)) == mdcn.MDCN_E_DEVICE                 # one pool
    assert call(dims(same), dst=at(0) + 544) == mdcn.MDCN_E_ALIAS
    assert call(dims(good[:1] + [0] + good[2:]), a=None, b=None) == mdcn.MDCN_OK
    assert call(dims(good)) == mdcn.MDCN_E_DEVICE


# ---------------------------------------------------------------- the binding

def test_the_binding_wants_device_tensors(cache):
    k = torch.zeros(4, 2, 64)
    pool = torch.zeros(3, cache.page_bytes, dtype=torch.uint8)
    table = torch.zeros(1, 3, dtype=torch.int32)
    used, cu = torch.tensor([4], dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)
    att = A.mdcn_attention_create(4, 2, 64, True)
    for call in (lambda: K.store(cache, pool, k, k, table, used, cu),
                 lambda: K.load(cache, pool, table, used, cu, 4, torch.float32),
                 lambda: K.attend(att, cache, torch.zeros(4, 4, 64), pool, table, used, cu),
                 lambda: K.fork_pages(pool, table, used, torch.zeros(3, dtype=torch.int32), 32),
                 lambda: K.compact_pages(pool, table, torch.zeros(3, dtype=torch.int32)),
                 lambda: K.copy_pages(pool, pool, used, used)):
        with pytest.raises(mdcn.MdcnError) as e:
            call()
        assert e.value.status == mdcn.MDCN_E_NULL
