"""Workspaces that the caller gives."""
import pytest
import torch

from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from modulated_deformable_convolution_amd import mdcn
from test_gpu_attention import ints, rand

pytestmark = pytest.mark.gpu
ensure_built()


def test_workspaces_of_the_caller():
    """Used where they are on the tensors' device and whole, refused elsewhere before any launch."""
    op, rot = A.mdcn_attention_create(2, 1, 64, True), A.mdcn_rotary_create(64, [32])
    q, k = rand(2, 2, 64, seed=1, dtype=torch.float16).cuda(), \
        rand(5000, 1, 64, seed=2, dtype=torch.float16).cuda()
    cq, ck, pos = ints([0, 2]), ints([0, 5000]), ints([[0, 1]])
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    out, lse = A.attend(op, q, k, k, cq, ck)
    n = 1 << 25
    calls = [lambda x: A.attend(op, q, k, k, cq, ck, workspace=x)[0],
             lambda x: A.attend_backward(op, q, k, k, out, lse, q, cq, ck, workspace=x)["k"],
             lambda x: A.norm_rotate_backward(rot, q, k[:2], pos, w, w, q, k[:2], workspace=x)["q"]]
    for call in calls:
        want = call(None)
        assert torch.equal(call(torch.empty(n, dtype=torch.uint8, device="cuda")), want)
        assert torch.equal(call(torch.empty(n // 4, device="cuda")), want)
        for bad in (torch.empty(n, dtype=torch.uint8),
                    torch.empty(n, 2, dtype=torch.uint8, device="cuda")[:, 0],
                    torch.empty(16, dtype=torch.uint8, device="cuda")):
            with pytest.raises(mdcn.MdcnError) as e:
                call(bad)
            assert e.value.status == mdcn.MDCN_E_WORKSPACE
