"""Attention on the GPU where it can go wrong."""
import pytest

import attention_reference as R
from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from test_gpu_attention import DTYPES, attend_case, ints, within

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
