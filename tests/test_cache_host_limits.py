"""Sizes of the cache and page entry points that are past what the library counts with: refused on
the host (the pointers here are addresses that nothing reads)."""
import ctypes

import pytest

from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from modulated_deformable_convolution_amd import cache as K
from modulated_deformable_convolution_amd import mdcn
from test_cache_host import STEP, at, attended, dims

ensure_built()


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("heads,batch,tokens,width,taken", [
    (16, 1 << 24, 1 << 24, 1, False),                # 2.8e8 items
    (16, 1 << 24, 1 << 24, 1 << 26, False),
    (16, 1 << 24, 100, 1 << 26, True),               # queries of 100 sequences at most
    (16, 1 << 22, 1 << 22, 1 << 20, True),
    (16, 1 << 24, 1 << 10, 1, True),
    (65536, 1 << 11, 1 << 11, 1, True),
    (65536, 1 << 12, 1 << 12, 1, False),
    (65536, 1, 1 << 20, 1, False),                   # many rows of one sequence
    (64, 1, 1 << 29, 1, False),
    (64, 1, 1 << 24, 1, True),
    (64, 0, 1 << 29, 1, True),                       # tokens of no sequence
])
def test_more_work_than_31_bits_count(dtype, heads, batch, tokens, width, taken):
    att, op = A.mdcn_attention_create(heads, heads, 8, True), K.mdcn_cache_create(heads, 8, 16)
    d = dims([batch, tokens, 1, op.page_bytes, width, width, heads * 8, 8, heads * 8, 8])
    lib, n, buf = mdcn.library(), ctypes.c_size_t(), ctypes.create_string_buffer(256)
    want = mdcn.MDCN_OK if taken else mdcn.MDCN_E_SHAPE
    assert lib.mdcn_cache_attend_workspace_bytes(att.handle, op.handle, dtype, d, ctypes.byref(n)) == want
    assert lib.mdcn_describe_cache_attend(att.handle, op.handle, dtype, d, buf, 256) == want
    if not taken:
        assert attended(att.handle, op.handle, d, dtype) == want


@pytest.mark.parametrize("pages,stride,taken", [
    (1 << 24, 1 << 40, False), ((1 << 24) + 1, 1 << 40, False), ((1 << 31) - 1, 1 << 33, False),
    ((1 << 31) - 1, 1 << 29, True), ((1 << 20) - 1, 1 << 40, True),
])
def test_pools_whose_bytes_64_bits_do_not_count(pages, stride, taken):
    """Their extent decides what may overlap what."""
    lib, n = mdcn.library(), ctypes.c_size_t()
    want = mdcn.MDCN_OK if taken else mdcn.MDCN_E_SHAPE
    fork, compact = [1, pages, 16, stride, 0, 16, 4, 6, 5], [1, pages, 16, stride, 0, 4, 5]
    assert lib.mdcn_pages_fork_workspace_bytes(dims(fork), ctypes.byref(n)) == want
    assert lib.mdcn_pages_compact_workspace_bytes(dims(compact), ctypes.byref(n)) == want
    copy = dims([1, 7, 16, pages, stride, 0, 30, 16, 0])
    st = lib.mdcn_pages_copy(copy, at(0), at(0) - STEP, at(0) - 2 * STEP, at(0) - 3 * STEP, None)
    assert st == (mdcn.MDCN_E_DEVICE if taken else want)
