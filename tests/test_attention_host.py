"""Host checks of the attention entry points: what they refuse, before any GPU
is asked for anything (the pointers here are addresses that nothing reads)."""
import ctypes

import pytest
import torch

from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from modulated_deformable_convolution_amd import mdcn

ensure_built()
BASE = 1 << 20


def dims(*v):
    return (ctypes.c_int64 * len(v))(*v)


def buffers(n, step=1 << 16):
    return [BASE + i * step for i in range(n)]


@pytest.mark.parametrize("kw", [
    dict(dim=0), dict(dim=7), dict(dim=258), dict(axes=[]), dict(axes=[5]), dict(axes=[0, 0]),
    dict(axes=[-1, 2]), dict(axes=[1] * 9, dim=64), dict(base=0.0), dict(base=-2.0),
    dict(base=float("nan")), dict(base=float("inf")), dict(axes=[2 ** 30, 2 ** 30, 2 ** 30]),
])
def test_rotary_create_refuses(kw):
    with pytest.raises(mdcn.MdcnError) as e:
        A.mdcn_rotary_create(**{**dict(dim=8, axes=[2, 2]), **kw})
    assert e.value.status == mdcn.MDCN_E_ATTR


@pytest.mark.parametrize("kw", [
    dict(q_heads=0), dict(k_heads=0), dict(q_heads=6), dict(dim=0), dict(dim=12), dict(dim=136),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
])
def test_attention_create_refuses(kw):
    with pytest.raises(mdcn.MdcnError) as e:
        A.mdcn_attention_create(**{**dict(q_heads=8, k_heads=4, dim=64, causal=True), **kw})
    assert e.value.status == mdcn.MDCN_E_ATTR


def rotate_status(d, dtype=0, q=BASE, k=BASE + 4096, pos=BASE + 8192, qo=BASE + 16384,
                  ko=BASE + 32768, op=None):
    op = op or A.mdcn_rotary_create(8, [2, 2])
    return mdcn.library().mdcn_rotate(op.handle, dtype, d, q, k, pos, 0, qo, ko, None)


GOOD_ROT = (10, 2, 1, 10, 16, 8, 8, 8, 16, 8, 8, 8)


@pytest.mark.parametrize("change,code", [
    ({0: -1}, "SHAPE"), ({1: -1}, "SHAPE"), ({1: 0, 2: 0}, "SHAPE"), ({3: 9}, "SHAPE"),
    ({4: -16}, "SHAPE"), ({5: -8}, "SHAPE"), ({4: 1 << 23}, "SHAPE"), ({8: 15}, "ALIAS"),
    ({9: 7}, "ALIAS"), ({8: 0}, "ALIAS"), ({0: 1 << 31}, "SHAPE"),
])
def test_rotate_refuses_dims(change, code):
    d = list(GOOD_ROT)
    for i, v in change.items():
        d[i] = v
    assert rotate_status(dims(*d)) == getattr(mdcn, "MDCN_E_" + code)


def test_rotate_refuses_pointers():
    d = dims(*GOOD_ROT)
    assert rotate_status(d, dtype=3) == mdcn.MDCN_E_DTYPE
    assert rotate_status(d, q=0) == mdcn.MDCN_E_NULL
    assert rotate_status(d, pos=0) == mdcn.MDCN_E_NULL
    assert rotate_status(d, ko=0) == mdcn.MDCN_E_NULL
    assert rotate_status(d, qo=BASE + 4) == mdcn.MDCN_E_ALIAS           # shifted over its input
    assert rotate_status(d, qo=BASE + 2) == mdcn.MDCN_E_SHAPE           # not aligned to a value
    assert rotate_status(d, qo=BASE + 4096) == mdcn.MDCN_E_ALIAS        # q's output over k
    assert rotate_status(d, ko=BASE + 16384) == mdcn.MDCN_E_ALIAS       # both outputs in one place
    assert rotate_status(d, qo=BASE + 8192) == mdcn.MDCN_E_ALIAS        # over the positions
    assert rotate_status(None) == mdcn.MDCN_E_NULL
    assert mdcn.library().mdcn_rotate(None, 0, d, BASE, BASE, BASE, 0, BASE, BASE,
                                      None) == mdcn.MDCN_E_NULL


@pytest.mark.skipif(torch.cuda.is_available(), reason="would run on the GPU")
def test_accepted_calls_reach_the_device_check():
    ok = mdcn.MDCN_E_DEVICE
    assert rotate_status(dims(*GOOD_ROT)) == ok
    assert rotate_status(dims(*GOOD_ROT), qo=BASE, ko=BASE + 4096) == ok      # in place
    # queries and keys as slices of one projection's rows, turned in place
    d = dims(10, 2, 1, 10, 24, 8, 24, 8, 24, 8, 24, 8)
    assert rotate_status(d, q=BASE, k=BASE + 64, qo=BASE, ko=BASE + 64) == ok
    # no keys
    assert rotate_status(dims(10, 2, 0, 10, 16, 8, 0, 0, 16, 8, 0, 0), k=0, ko=0) == ok
    # no tokens: nothing to do, no device needed
    assert rotate_status(dims(0, 2, 1, 0, 16, 8, 8, 8, 16, 8, 8, 8), q=0, k=0, pos=0, qo=0,
                         ko=0) == mdcn.MDCN_OK
    assert attend_status() == ok
    assert attend_status(q_tokens=0) == mdcn.MDCN_OK
    assert backward_status() == ok


def attend_status(dtype=2, q_tokens=300, change={}, ptr={}, ws=1 << 26):
    op = A.mdcn_attention_create(4, 2, 64, True)
    d = [3, q_tokens, 200, 256, 64, 128, 64, 128, 64, 256, 64]
    for i, v in change.items():
        d[i] = v
    names = ["q", "k", "v", "cu_q", "cu_k", "used", "out", "lse", "ws"]
    p = dict(zip(names, buffers(9, 1 << 24)))
    p.update(ptr)
    return mdcn.library().mdcn_attend(op.handle, dtype, dims(*d), *[p[n] for n in names], ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), "DTYPE"), (dict(change={0: -1}), "SHAPE"), (dict(change={1: -1}), "SHAPE"),
    (dict(change={2: -5}), "SHAPE"), (dict(change={3: 260}), "SHAPE"),
    (dict(change={6: 60}), "SHAPE"), (dict(change={3: -256}), "SHAPE"),
    (dict(change={5: 1 << 23}), "SHAPE"), (dict(change={5: 0}), "SHAPE"),
    (dict(change={7: 56}), "SHAPE"), (dict(change={9: 128}), "ALIAS"),
    (dict(ptr={"q": BASE + 2}), "SHAPE"), (dict(ptr={"k": BASE + 8 + (1 << 24)}), "SHAPE"),
    (dict(ptr={"q": 0}), "NULL"), (dict(ptr={"v": 0}), "NULL"), (dict(ptr={"cu_q": 0}), "NULL"),
    (dict(ptr={"cu_k": 0}), "NULL"), (dict(ptr={"lse": 0}), "NULL"),
    (dict(ptr={"out": BASE}), "ALIAS"), (dict(ptr={"lse": BASE}), "ALIAS"),
    (dict(q_tokens=3, change={2: 60000}, ws=16), "WORKSPACE"),
    (dict(q_tokens=3, change={2: 60000}, ptr={"ws": 0}), "WORKSPACE"),
    (dict(q_tokens=3, change={2: 60000}, ptr={"ws": BASE}), "ALIAS"),
])
def test_attend_refuses(kw, code):
    assert attend_status(**kw) == getattr(mdcn, "MDCN_E_" + code)


def backward_status(dtype=2, change={}, ptr={}, ws=1 << 22):
    op = A.mdcn_attention_create(4, 2, 64, True)
    d = [3, 300, 200, 256, 64, 128, 64, 128, 64, 256, 64, 256, 64, 256, 64, 128, 64, 128, 64]
    for i, v in change.items():
        d[i] = v
    names = ["q", "k", "v", "out", "lse", "go", "cu_q", "cu_k", "used", "gq", "gk", "gv", "ws"]
    p = dict(zip(names, buffers(13, 1 << 24)))
    p.update(ptr)
    return mdcn.library().mdcn_attend_backward(op.handle, dtype, dims(*d), *[p[n] for n in names],
                                               ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), "DTYPE"), (dict(change={11: 4}), "SHAPE"), (dict(change={13: 128}), "ALIAS"),
    (dict(ptr={"go": 0}), "NULL"), (dict(ptr={"gv": 0}), "NULL"), (dict(ptr={"lse": 0}), "NULL"),
    (dict(ptr={"gq": BASE}), "ALIAS"), (dict(ptr={"gk": BASE + 11 * (1 << 24)}), "ALIAS"),
    (dict(ptr={"ws": 0}), "WORKSPACE"), (dict(ws=100), "WORKSPACE"),
    (dict(ptr={"ws": BASE}), "ALIAS"),
])
def test_attend_backward_refuses(kw, code):
    assert backward_status(**kw) == getattr(mdcn, "MDCN_E_" + code)


def norm_backward_status(change={}, ptr={}, ws=1 << 22, eps=1e-6):
    op = A.mdcn_rotary_create(8, [2, 2])
    d = [10, 2, 1, 10] + [16, 8, 8, 8] * 3
    for i, v in change.items():
        d[i] = v
    names = ["q", "k", "pos", "qg", "kg", "gq", "gk", "dq", "dk", "dqg", "dkg", "ws"]
    p = dict(zip(names, buffers(12, 1 << 23)))
    p.update(ptr)
    v = [p[n] for n in names]
    return mdcn.library().mdcn_norm_rotate_backward(op.handle, 0, dims(*d), *v[:5], eps, *v[5:], ws,
                                                    None)


@pytest.mark.parametrize("kw,code", [
    (dict(eps=-1.0), "ATTR"), (dict(eps=float("nan")), "ATTR"), (dict(ws=10), "WORKSPACE"),
    (dict(ptr={"ws": 0}), "WORKSPACE"), (dict(ptr={"dqg": 0}), "NULL"),
    (dict(ptr={"kg": 0}), "NULL"), (dict(ptr={"dq": BASE}), "ALIAS"),
    (dict(ptr={"dqg": BASE}), "ALIAS"), (dict(ptr={"dqg": BASE + 3 * (1 << 23)}), "ALIAS"),
    (dict(change={12: 8}), "ALIAS"),
])
def test_norm_rotate_backward_refuses(kw, code):
    assert norm_backward_status(**kw) == getattr(mdcn, "MDCN_E_" + code)


def test_host_tensors_are_refused():
    op = A.mdcn_rotary_create(8, [4])
    x, pos = torch.zeros(3, 2, 8), torch.zeros(1, 3, dtype=torch.int32)
    gain = torch.ones(8)
    att = A.mdcn_attention_create(2, 2, 8, True)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    for call in (lambda: A.rotate(op, x, x, pos), lambda: A.rotate_backward(op, x, x, pos),
                 lambda: A.norm_rotate(op, x, x, pos, gain, gain),
                 lambda: A.norm_rotate_backward(op, x, x, pos, gain, gain, x, x),
                 lambda: A.attend(att, x, x, x, cu, cu),
                 lambda: A.attend_backward(att, x, x, x, x, torch.zeros(2, 3), x, cu, cu)):
        with pytest.raises(mdcn.MdcnError) as e:
            call()
        assert e.value.status == mdcn.MDCN_E_NULL


def test_workspace_sizes():
    att = A.mdcn_attention_create(8, 2, 128, True)
    n = ctypes.c_size_t(7)
    lib = mdcn.library()
    few, many = dims(4, 4, 4096, *[0] * 8), dims(1, 4096, 4096, *[0] * 8)
    assert lib.mdcn_attend_workspace_bytes(att.handle, 2, few, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.mdcn_attend_workspace_bytes(att.handle, 2, many, ctypes.byref(n)) == 0
    assert n.value == 0
    assert lib.mdcn_attend_workspace_bytes(att.handle, 9, many,
                                           ctypes.byref(n)) == mdcn.MDCN_E_DTYPE
    assert lib.mdcn_attend_workspace_bytes(att.handle, 2, many, None) == mdcn.MDCN_E_NULL
