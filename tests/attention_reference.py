"""Plain 64-bit forms of the attention operators (CPU) with bounds on how far
a kernel that follows their rounding rules may be off.

The bounds count roundings: u = eps(T) / 2 relative for each rounding to the
tensors' type T (outputs, probabilities and score gradients), and 2^-24 for each
fp32 operation along a value's chain of sums.
"""
import math

import torch

E32 = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half a step below the normal numbers."""
    return torch.finfo(dtype).smallest_normal * unit(dtype)


# ---------------------------------------------------------------- rotary positions

def angles(axes, base, round_robin, per_axis, positions):
    """[tokens][pairs] angles."""
    order = []
    if round_robin:
        for j in range(max(axes)):
            order += [(a, j) for a, n in enumerate(axes) if j < n]
    else:
        for a, n in enumerate(axes):
            order += [(a, j) for j in range(n)]
    cols = []
    for i, (a, j) in enumerate(order):
        e = j / axes[a] if per_axis else i / len(order)
        cols.append(positions[a].double() * base ** -e)
    return torch.stack(cols, 1)


def turn(x, theta, adjacent, absolute=False):
    """x [tokens, heads, dim] turned; with absolute, |a||cos| + |b||sin| sums' upper
    bound |a| + |b| of every output."""
    p = theta.shape[1]
    x = x.clone()
    lo, hi = (slice(0, 2 * p, 2), slice(1, 2 * p, 2)) if adjacent else (slice(0, p), slice(p, 2 * p))
    a, b = x[..., lo].clone(), x[..., hi].clone()
    if absolute:
        x = x.abs()
        x[..., lo] = x[..., hi] = a.abs() + b.abs()
        return x
    c, s = theta.cos()[:, None], theta.sin()[:, None]
    x[..., lo], x[..., hi] = a * c - b * s, a * s + b * c
    return x


def rotate(x, theta, adjacent, dtype):
    """(value, bound)"""
    x = x.double()
    y = turn(x, theta, adjacent)
    return y, unit(dtype) * y.abs() + 8 * E32 * turn(x, theta, adjacent, True) + tiny(dtype)


def norm_rotate(x, gain, eps, theta, adjacent, dtype):
    x, gain = x.double(), gain.double()
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gain
    y = turn(n, theta, adjacent)
    d = x.shape[-1]
    return y, unit(dtype) * y.abs() + (d / 2 + 16) * E32 * turn(n, theta, adjacent, True) + \
        tiny(dtype)


def norm_rotate_backward(x, gain, eps, theta, adjacent, gy, dtype):
    """((dx, bound), (dgain, bound))"""
    x, gain, gy = x.double(), gain.double(), gy.double()
    inv = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    n = x * inv
    g = turn(gy, -theta, adjacent)
    g_abs = turn(gy, theta, adjacent, True)
    h = g * gain
    dx = inv * (h - n * (h * n).mean(-1, keepdim=True))
    d = x.shape[-1]
    mag = inv * (g_abs * gain.abs() + n.abs() * (g_abs * gain.abs() * n.abs()).mean(-1, keepdim=True))
    dgain = (g * n).sum((0, 1))
    terms = x.shape[0] * x.shape[1]
    mag_gain = (g_abs * n.abs()).sum((0, 1))
    return ((dx, unit(dtype) * dx.abs() + (2 * d + 32) * E32 * mag + tiny(dtype)),
            (dgain, unit(dtype) * dgain.abs() + (terms + d + 32) * E32 * mag_gain + tiny(dtype)))


# ---------------------------------------------------------------- attention

def visible(lq, lk, causal):
    i, j = torch.arange(lq)[:, None], torch.arange(lk)[None]
    return (j <= i + lk - lq) if causal else torch.ones(lq, lk, dtype=torch.bool)


def attend(q, k, v, cu_q, cu_k, used, causal, scale, dtype, grad_out=None):
    """A dict of (value, bound): out, lse and, with grad_out, q, k, v.  Tokens that
    belong to no sequence keep NaN values."""
    q, k, v = q.double(), k.double(), v.double()
    go = None if grad_out is None else grad_out.double()
    tq, hq, d = q.shape
    hk = k.shape[1]
    u = unit(dtype)
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.float64)  # noqa: E731
    r = {"out": (nan(tq, hq, d), nan(tq, hq, d)), "lse": (nan(hq, tq), nan(hq, tq))}
    if go is not None:
        r.update(q=(nan(tq, hq, d), nan(tq, hq, d)), k=(nan(*k.shape), nan(*k.shape)),
                 v=(nan(*k.shape), nan(*k.shape)))
    for b in range(len(cu_q) - 1):
        qs = slice(cu_q[b], cu_q[b + 1])
        lq = cu_q[b + 1] - cu_q[b]
        lk = cu_k[b + 1] - cu_k[b] if used is None else used[b]
        ks = slice(cu_k[b], cu_k[b] + lk)
        if go is not None:
            for n in "kv":
                for x in r[n]:
                    x[cu_k[b]:cu_k[b + 1]] = 0.0
        see = visible(lq, lk, causal)
        for h in range(hq):
            n = h // (hq // hk)
            qh, kh, vh = q[qs, h], k[ks, n], v[ks, n]
            # hidden rows of k and v take no part at all
            s = torch.where(see, (qh @ kh.T) * scale, torch.tensor(-math.inf, dtype=torch.float64))
            s_abs = (qh.abs() @ kh.abs().T) * scale
            lse = torch.logsumexp(s, 1) if lk else nan(lq) * 0 - math.inf
            lse = torch.where(see.any(1), lse, torch.tensor(-math.inf, dtype=torch.float64))
            p = torch.where(see, (s - lse[:, None]).exp(), torch.tensor(0.0, dtype=torch.float64))
            # a score's fp32 error, twice for score and maximum, and exp's
            top = torch.where(see, s_abs, torch.zeros_like(s_abs)).amax(1) if lk else \
                torch.zeros(lq, dtype=torch.float64)
            ds_err = ((2 * d + 16) * E32 * top + 16 * E32)[:, None]
            sum_err = lk * E32
            vz = torch.where(vh.isfinite(), vh, torch.zeros_like(vh))
            o = _product(p, vh, see)
            o_err = u * o.abs() + (u + 2 * ds_err + 2 * sum_err) * (p @ vz.abs()) + \
                tiny(dtype) * (1 + lk)
            r["out"][0][qs, h], r["out"][1][qs, h] = o, o_err
            r["lse"][0][h, qs] = lse
            r["lse"][1][h, qs] = ds_err[:, 0] + sum_err + 4 * E32 * lse.abs().nan_to_num(0, 0, 0)
            if go is None:
                continue
            g = go[qs, h]
            lse_err = r["lse"][1][h, qs][:, None]
            p_err = (u + 2 * ds_err + 2 * lse_err) * p + tiny(dtype)
            p_err = torch.where(see, p_err, torch.zeros_like(p_err))
            r["v"][0][ks, n] += p.T @ g
            r["v"][1][ks, n] += (p_err + (lq * (hq // hk)) * E32 * p).T @ g.abs()
            dp = g @ vh.T
            delta = (g * o).sum(1, keepdim=True)
            ds = p * (dp - delta)
            diff_err = 2 * d * E32 * (g.abs() @ vh.abs().T) + \
                (g.abs() * (o_err + d * E32 * o.abs())).sum(1, keepdim=True)
            ds_e = u * ds.abs() + (p_err - u * p).clamp(min=0) * (dp - delta).abs() + p * diff_err \
                + 4 * E32 * ds.abs() + tiny(dtype)
            ds_e = torch.where(see, ds_e, torch.zeros_like(ds_e))
            r["q"][0][qs, h] = ds @ kh * scale
            r["q"][1][qs, h] = (ds_e + lk * E32 * ds.abs()) @ kh.abs() * scale
            r["k"][0][ks, n] += ds.T @ qh * scale
            r["k"][1][ks, n] += (ds_e + (lq * (hq // hk)) * E32 * ds.abs()).T @ qh.abs() * scale
    if go is not None:
        for n in "qkv":
            r[n][1].add_(u * r[n][0].abs() + tiny(dtype))
    return r


def _product(p, v, see):
    """sum over the visible keys of p v; hidden rows of v are not touched."""
    if v.isfinite().all():
        return p @ v
    return torch.stack([sum((p[i, j] * v[j] for j in range(v.shape[0]) if see[i, j]),
                            torch.zeros(v.shape[1], dtype=torch.float64)) for i in range(p.shape[0])])
