"""The 64-bit reference of the attention operators against independent routes:
complex rotation, central differences, softmax on dense masks."""
import math

import pytest
import torch

import attention_reference as R


def rand(*shape, seed=0):
    return torch.randn(*shape, dtype=torch.float64, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("adjacent", [False, True])
def test_turn_is_a_complex_product(adjacent):
    x = rand(3, 2, 10)
    theta = rand(3, 4, seed=1)
    y = R.turn(x, theta, adjacent)
    for t in range(3):
        for i in range(4):
            a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + 4)
            z = torch.complex(x[t, :, a], x[t, :, b]) * complex(math.cos(theta[t, i]),
                                                               math.sin(theta[t, i]))
            assert torch.allclose(y[t, :, a], z.real) and torch.allclose(y[t, :, b], z.imag)
    assert torch.equal(y[..., 8:], x[..., 8:])


def test_angle_orders():
    pos = torch.tensor([[2, 3], [5, 7], [11, 13]])
    th = R.angles([2, 1, 3], 100.0, True, False, pos)
    owners = [0, 1, 2, 0, 2, 2]
    for i, a in enumerate(owners):
        assert torch.allclose(th[:, i], pos[a].double() * 100.0 ** (-i / 6))
    th = R.angles([2, 1, 3], 100.0, False, True, pos)
    for i, (a, j, n) in enumerate([(0, 0, 2), (0, 1, 2), (1, 0, 1), (2, 0, 3), (2, 1, 3), (2, 2, 3)]):
        assert torch.allclose(th[:, i], pos[a].double() * 100.0 ** (-j / n))


def difference(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_norm_rotate_gradients_match_differences():
    x, gain, gy = rand(4, 3, 12), 1 + 0.2 * rand(12, seed=1), rand(4, 3, 12, seed=2)
    theta = rand(4, 4, seed=3)
    (dx, _), (dg, _) = R.norm_rotate_backward(x, gain, 1e-3, theta, False, gy, torch.float32)
    loss = lambda a, b: (R.norm_rotate(a, b, 1e-3, theta, False, torch.float32)[0] * gy).sum()  # noqa
    for seed in range(3):
        d = rand(4, 3, 12, seed=10 + seed)
        assert abs(difference(lambda v: loss(v, gain), x, d) - (dx * d).sum()) < 1e-7
        d = rand(12, seed=20 + seed)
        assert abs(difference(lambda v: loss(x, v), gain, d) - (dg * d).sum()) < 1e-7


@pytest.mark.parametrize("causal", [False, True])
def test_attention_gradients_match_differences(causal):
    cu_q, cu_k = [0, 5, 5, 6, 13], [0, 3, 5, 5, 14]
    q, k, v, go = rand(13, 4, 8), rand(14, 2, 8, seed=1), rand(14, 2, 8, seed=2), rand(13, 4, 8, seed=3)
    run = lambda q, k, v: R.attend(q, k, v, cu_q, cu_k, None, causal, 0.4, torch.float32, go)  # noqa
    g = run(q, k, v)
    loss = lambda q, k, v: (run(q, k, v)["out"][0] * go).sum()  # noqa: E731
    for seed in range(2):
        d = rand(13, 4, 8, seed=30 + seed)
        assert abs(difference(lambda x: loss(x, k, v), q, d) - (g["q"][0] * d).sum()) < 1e-7
        d = rand(14, 2, 8, seed=40 + seed)
        assert abs(difference(lambda x: loss(q, x, v), k, d) - (g["k"][0] * d).sum()) < 1e-7
        assert abs(difference(lambda x: loss(q, k, x), v, d) - (g["v"][0] * d).sum()) < 1e-7


def test_empty_rows_and_hidden_values():
    q, k, v = rand(5, 2, 8), rand(3, 1, 8, seed=1), rand(3, 1, 8, seed=2)
    r = R.attend(q, k, v, [0, 5], [0, 3], None, True, 0.3, torch.float32)
    assert (r["out"][0][:2] == 0).all() and (r["lse"][0][:, :2] == -math.inf).all()
    w = v.clone()
    w[2] = math.nan
    s = R.attend(q, k, w, [0, 5], [0, 3], None, True, 0.3, torch.float32)
    assert torch.allclose(s["out"][0][:4], r["out"][0][:4]) and s["out"][0][4].isnan().all()
    p = torch.softmax((q[4, 0] @ k[:, 0].T) * 0.3, 0)
    assert torch.allclose(r["out"][0][4, 0], p @ v[:, 0])
