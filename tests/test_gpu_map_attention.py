"""The operators run together (map_attention), against 64-bit arithmetic."""
import pytest
import torch

import attention_reference as R
from helpers import ensure_built
from modulated_deformable_convolution_amd import map_attention as M

pytestmark = pytest.mark.gpu
ensure_built()


def test_map_attention_gradients_against_differences():
    """fp32 gradients of a whole layer against central differences of its 64-bit form."""
    sizes = [(5, 6), (3, 1), (1, 1), (9, 4)]
    layer = M.MapAttention(16, 4, 2, 32, dtype=torch.float32, seed=1)
    plan = layer.plan(sizes)
    gen = torch.Generator().manual_seed(2)
    n = sum(h * w for h, w in sizes)
    tokens = torch.randn(n, 16, generator=gen)
    grad = torch.randn(n, 128, generator=gen)
    out, saved = layer.forward(tokens.cuda(), plan)
    got = {k: v.double().cpu() for k, v in layer.backward(grad.cuda(), saved).items()}
    ends = plan[1].tolist()
    theta = R.angles([8, 8], 100.0, False, False, plan[0].cpu())

    def value(x, w, gq, gk):
        qkv = (x @ w.t()).unflatten(1, (8, 32))
        q = R.norm_rotate(qkv[:, :4], gq, 1e-6, theta, False, torch.float32)[0]
        k = R.norm_rotate(qkv[:, 4:6], gk, 1e-6, theta, False, torch.float32)[0]
        return R.attend(q, k, qkv[:, 6:], ends, ends, None, False, 32 ** -0.5,
                        torch.float32)["out"][0].flatten(1)

    args = [tokens.double(), layer.weight.double().cpu(), torch.ones(32, dtype=torch.float64),
            torch.ones(32, dtype=torch.float64)]
    want = value(*args)
    # a few hundred fp32 roundings in a row, relative to the tensors' size
    assert float((out.double().cpu() - want).norm() / want.norm()) < 512 * R.E32
    for i, name in enumerate(("tokens", "weight", "q_gain", "k_gain")):
        d = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        ends_of = [[a + s * h * d if j == i else a for j, a in enumerate(args)] for s in (1, -1)]
        diff = float(((value(*ends_of[0]) - value(*ends_of[1])) * grad.double()).sum()) / (2 * h)
        have = float((got[name] * d).sum())
        assert abs(have - diff) <= 512 * R.E32 * float(got[name].norm() * d.norm()) + 1e-7, name


def test_decoding_equals_the_whole_sequence():
    """Steps against the cache give what one causal pass over the sequences gives."""
    gen = torch.Generator().manual_seed(3)
    lengths, steps = [5, 40, 1], 6
    x = [torch.randn(n + steps, 32, generator=gen).half() for n in lengths]
    dec = M.Decoder(32, 4, 2, 64, batch=3, room=64)
    got = [list(dec.prompt(torch.cat([t[:n] for t, n in zip(x, lengths)]).cuda(), lengths)
                .split(lengths))]
    for i in range(steps):
        got.append(list(dec.step(torch.stack([t[n + i] for t, n in zip(x, lengths)]).cuda())
                        .split([1] * 3)))
    whole = M.Decoder(32, 4, 2, 64, batch=3, room=64)
    full = [n + steps for n in lengths]
    want = whole.prompt(torch.cat(x).cuda(), full).split(full)
    for b in range(3):
        have = torch.cat([g[b] for g in got])
        # the same numbers in another order of sums: a few steps of fp16
        assert float((have - want[b]).abs().max()) <= 8 * R.unit(torch.float16) * \
            float(want[b].abs().max())
    assert dec.used.tolist() == full


def test_example_runs(capsys):
    M.main()
    assert "decoded 4 tokens" in capsys.readouterr().out
