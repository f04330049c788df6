"""More that the attention entry points refuse or take, before any GPU is asked for
anything (the pointers here are addresses that nothing reads)."""
import pytest
import torch

from helpers import ensure_built
from modulated_deformable_convolution_amd import attention as A
from modulated_deformable_convolution_amd import mdcn
from test_attention_host import attend_status, backward_status, dims, rotate_status

ensure_built()
BASE, STEP = 1 << 20, 1 << 24
# where test_attention_host puts the buffers
FORWARD = {n: BASE + i * STEP for i, n in enumerate(
    ["q", "k", "v", "cu_q", "cu_k", "used", "out", "lse", "ws"])}
BACKWARD = {n: BASE + i * STEP for i, n in enumerate(
    ["q", "k", "v", "out", "lse", "go", "cu_q", "cu_k", "used", "gq", "gk", "gv", "ws"])}
FEW = dict(q_tokens=3, change={2: 60000}, ws=9 << 20)        # few rows, many keys: with a workspace


@pytest.mark.parametrize("other", ["cu_q", "cu_k", "used"])
@pytest.mark.parametrize("kw", [{}, FEW], ids=["tiles", "split"])
def test_lse_over_what_the_forward_reads(kw, other):
    assert attend_status(ptr={"lse": FORWARD[other]}, **kw) == mdcn.MDCN_E_ALIAS
    assert attend_status(ptr={"lse": FORWARD[other] - 4}, **kw) == mdcn.MDCN_E_ALIAS


@pytest.mark.parametrize("other", ["cu_q", "cu_k", "used", "lse"])
def test_forward_workspace_over_other_buffers(other):
    assert attend_status(ptr={"ws": FORWARD[other]}, **FEW) == mdcn.MDCN_E_ALIAS
    assert attend_status(ptr={"ws": FORWARD[other] - 256}, **FEW) == mdcn.MDCN_E_ALIAS


@pytest.mark.parametrize("other", ["cu_q", "cu_k", "used", "lse"])
def test_backward_workspace_over_other_buffers(other):
    assert backward_status(ptr={"ws": BACKWARD[other]}) == mdcn.MDCN_E_ALIAS
    assert backward_status(ptr={"ws": BACKWARD[other] - 256}) == mdcn.MDCN_E_ALIAS


@pytest.mark.skipif(torch.cuda.is_available(), reason="would run on the GPU")
def test_buffers_side_by_side_are_taken():
    """Buffers of one arena that touch and do not overlap."""
    lse = FORWARD["cu_q"] - 4 * 300 * 4
    assert attend_status(ptr={"lse": lse}) == mdcn.MDCN_E_DEVICE
    assert attend_status(ptr={"lse": FORWARD["cu_q"] + 16}) == mdcn.MDCN_E_DEVICE
    assert attend_status(**FEW) == mdcn.MDCN_E_DEVICE
    # the tile kernel has no workspace: whatever is given is not looked at
    assert attend_status(ptr={"ws": FORWARD["cu_q"]}) == mdcn.MDCN_E_DEVICE
    assert backward_status(ptr={"ws": BACKWARD["cu_q"] - (1 << 22)}) == mdcn.MDCN_E_DEVICE
    assert backward_status(ptr={"used": 0}) == mdcn.MDCN_E_DEVICE


@pytest.mark.skipif(torch.cuda.is_available(), reason="would run on the GPU")
def test_empty_views_share_nothing():
    """No keys: their pointers may lie anywhere, inside an output too."""
    inside = {"k": FORWARD["out"] + 512, "v": FORWARD["out"] + 1024}
    assert attend_status(change={2: 0}, ptr=inside) == mdcn.MDCN_E_DEVICE
    assert attend_status(change={2: 0}, ptr={"k": FORWARD["lse"] + 512}) == mdcn.MDCN_E_DEVICE
    assert attend_status(change={2: 200}, ptr=inside) == mdcn.MDCN_E_ALIAS


@pytest.mark.skipif(torch.cuda.is_available(), reason="would run on the GPU")
@pytest.mark.parametrize("tokens", [1, 10])
def test_rotation_in_place_of_queries_and_keys_that_alternate(tokens):
    """[tokens][heads][query, key, value][dim]: no value belongs to two views."""
    def status(q, k, q_out, k_out, heads=2, row=48):
        d = dims(tokens, heads, heads, tokens, row, 24, row, 24, row, 24, row, 24)
        return rotate_status(d, q=q, k=k, pos=BASE - 8192, qo=q_out, ko=k_out)
    key = BASE + 8 * 4
    assert status(BASE, key, BASE, key) == mdcn.MDCN_E_DEVICE
    assert status(BASE, key, key, BASE) == mdcn.MDCN_E_ALIAS              # exchanged
    assert status(BASE, key, BASE + 16 * 4, key) == mdcn.MDCN_E_DEVICE    # into the values' place
    assert status(BASE, key, BASE + 4 * 4, key) == mdcn.MDCN_E_ALIAS      # half of it
    assert status(BASE, key, BASE + 20 * 4, key) == mdcn.MDCN_E_ALIAS     # over the next head's
    assert status(BASE, key, BASE, BASE + 4 * 4) == mdcn.MDCN_E_ALIAS
    # rows whose stride the heads' does not divide
    assert status(BASE, key, BASE, key, row=50) == (
        mdcn.MDCN_E_ALIAS if tokens > 1 else mdcn.MDCN_E_DEVICE)


@pytest.mark.parametrize("bad", [
    torch.zeros(64, dtype=torch.uint8, device="meta"), torch.zeros(64, 2, dtype=torch.uint8)[:, 0],
    torch.zeros(64, dtype=torch.uint8).expand(2, 64),
])
def test_workspaces_elsewhere_are_refused(bad):
    """A workspace on another device, or with gaps, would be written past its memory."""
    like = torch.zeros(1)
    with pytest.raises(mdcn.MdcnError) as e:
        A._workspace_bytes("attend", bad, like)
    assert e.value.status == mdcn.MDCN_E_WORKSPACE
    assert A._workspace_bytes("attend", torch.zeros(64, dtype=torch.uint8), like) == 64
    assert A._workspace_bytes("attend", torch.zeros(3, 5), like) == 60
    assert A._workspace_bytes("attend", None, like) == 0


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Kernels are launched on the current device."""
    monkeypatch.setattr(A, "_current_device", lambda: 0)
    A._check_current("attend", 0)
    with pytest.raises(mdcn.MdcnError) as e:
        A._check_current("attend", 1)
    assert e.value.status == mdcn.MDCN_E_DEVICE


def test_descriptions():
    op, rot = A.mdcn_attention_create(32, 8, 128, True), A.mdcn_rotary_create(128, [64])
    assert A.describe_attend(op, torch.bfloat16, 4, 4096, 4096) == "tile rows=128 key_waves=1"
    assert A.describe_attend(op, torch.bfloat16, 48, 48, 48 * 8192).startswith("split unit=32 ")
    assert A.describe_rotate(rot, torch.float16, 1, 32, 8) == \
        "width=8 lanes=8 rounds=1 waves_per_token=5 backward_blocks=1"
    assert A.describe_rotate(rot, torch.float32, 0, 32, 8) == "nothing to do"
    for call in (lambda: A.describe_attend(op, torch.float16, -1, 1, 1),
                 lambda: A.describe_attend(op, torch.float64, 1, 1, 1),
                 lambda: A.describe_rotate(rot, torch.float16, -1, 1, 1),
                 lambda: A.describe_rotate(rot, torch.float16, 1, 0, 0)):
        with pytest.raises(mdcn.MdcnError):
            call()
