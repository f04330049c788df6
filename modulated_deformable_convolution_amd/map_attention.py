"""The operators together, as a detector and its captioner use them.

    python -m modulated_deformable_convolution_amd.map_attention

MapAttention attends over the maps that deformable convolutions produce: maps
of different sizes are packed as tokens, projected, normed and turned by their
row and column, and attended in full, each map by itself; its backward pass
gives the gradients of the tokens, the projection and the gains.  Decoder runs a
causal layer over growing sequences, one token of each at a time, against a
key/value cache.  The projections are plain torch products; everything else is
the library's kernels.
"""
from __future__ import annotations

import torch

from . import attention, mdcn


def _normal(gen, shape, dtype, scale):
    return (torch.randn(shape, generator=gen) * scale).to("cuda", dtype)


class _Layer:
    def __init__(self, channels, q_heads, k_heads, dim, axes, causal, base, dtype, seed):
        gen = torch.Generator().manual_seed(seed)
        self.q_heads, self.k_heads, self.dim = q_heads, k_heads, dim
        self.weight = _normal(gen, ((q_heads + 2 * k_heads) * dim, channels), dtype,
                              channels ** -0.5)
        self.q_gain, self.k_gain = (torch.ones(dim, dtype=dtype, device="cuda") for _ in range(2))
        self.rotary = attention.mdcn_rotary_create(dim, axes, base=base)
        self.attention = attention.mdcn_attention_create(q_heads, k_heads, dim, causal)

    def project(self, tokens):
        """Queries, keys and values as slices of one projection's output."""
        qkv = (tokens @ self.weight.t()).unflatten(1, (self.q_heads + 2 * self.k_heads, self.dim))
        return qkv.split((self.q_heads, self.k_heads, self.k_heads), 1)


class MapAttention(_Layer):
    """Full attention within each of several maps; rows and columns are the
    two axes of the positions."""

    def __init__(self, channels, q_heads, k_heads, dim, dtype=torch.float16, seed=0):
        super().__init__(channels, q_heads, k_heads, dim, [dim // 4, dim // 4], False, 100.0, dtype,
                         seed)

    @staticmethod
    def plan(sizes):
        """(positions, offsets) of maps of sizes [(height, width), ...]."""
        grid = [torch.stack(torch.meshgrid(torch.arange(h), torch.arange(w), indexing="ij")
                            ).flatten(1) for h, w in sizes]
        ends = torch.tensor([0] + [h * w for h, w in sizes]).cumsum(0)
        return torch.cat(grid, 1).to("cuda", torch.int32), ends.to("cuda", torch.int32)

    def forward(self, tokens, plan):
        """tokens [all pixels, channels] -> ([all pixels, q_heads * dim], what backward needs)."""
        positions, ends = plan
        q, k, v = self.project(tokens)
        q_turned, k_turned = attention.norm_rotate(self.rotary, q, k, positions, self.q_gain,
                                                   self.k_gain)
        out, lse = attention.attend(self.attention, q_turned, k_turned, v, ends, ends)
        return out.flatten(1), (tokens, plan, q, k, v, q_turned, k_turned, out, lse)

    def backward(self, grad, saved):
        """Gradients: a dict of tokens, weight, q_gain and k_gain."""
        tokens, (positions, ends), q, k, v, q_turned, k_turned, out, lse = saved
        a = attention.attend_backward(self.attention, q_turned, k_turned, v, out, lse,
                                      grad.unflatten(1, (self.q_heads, self.dim)), ends, ends)
        n = attention.norm_rotate_backward(self.rotary, q, k, positions, self.q_gain, self.k_gain,
                                           a["q"], a["k"])
        qkv = torch.cat((n["q"], n["k"], a["v"]), 1).flatten(1)
        return {"tokens": qkv @ self.weight, "weight": qkv.t() @ tokens, "q_gain": n["q_gain"],
                "k_gain": n["k_gain"]}


class Decoder(_Layer):
    """A causal layer with a cache of `room` tokens for each of `batch` sequences."""

    def __init__(self, channels, q_heads, k_heads, dim, batch, room, dtype=torch.float16, seed=0):
        super().__init__(channels, q_heads, k_heads, dim, [dim // 2], True, 10000.0, dtype, seed)
        self.batch, self.room = batch, room
        # keys and values that nobody has written yet are never read
        self.keys, self.values = (torch.empty((batch * room, k_heads, dim), dtype=dtype,
                                              device="cuda") for _ in range(2))
        self.used = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.longest = 0
        self.first = torch.arange(batch, device="cuda") * room
        self.new_ends = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
        self.cache_ends = self.new_ends * room

    def prompt(self, tokens, lengths):
        """Packed prompts (lengths: a list): fills the cache, returns the outputs."""
        if len(lengths) != self.batch or max(lengths) > self.room:
            raise ValueError("%d prompts of at most %d tokens" % (self.batch, self.room))
        steps = torch.cat([torch.arange(n) for n in lengths]).cuda()
        rows = torch.repeat_interleave(self.first, torch.tensor(lengths).cuda()) + steps
        ends = torch.tensor([0] + lengths).cumsum(0).to("cuda", torch.int32)
        q, k, v = self.project(tokens)
        q, k = attention.rotate(self.rotary, q, k, steps.to(torch.int32)[None])
        self.keys[rows], self.values[rows] = k, v
        self.used = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.longest = max(lengths)
        return attention.attend(self.attention, q, k, v, ends, ends)[0].flatten(1)

    def step(self, tokens):
        """The next token of every sequence, [batch, channels]."""
        if self.longest == self.room:
            raise ValueError("the cache is full")
        self.longest += 1
        q, k, v = self.project(tokens)
        q, k = attention.rotate(self.rotary, q, k, self.used[None])
        rows = self.first + self.used
        self.keys[rows], self.values[rows] = k, v
        self.used = self.used + 1
        return attention.attend(self.attention, q, self.keys, self.values, self.new_ends,
                                self.cache_ends, used_k=self.used)[0].flatten(1)


def main():
    gen = torch.Generator().manual_seed(0)
    channels, sizes = 64, [(40, 40), (24, 24), (7, 5)]
    conv = mdcn.mdcn_create(1, 1, 1, 1, 1)
    weight = _normal(gen, (channels, channels, 3, 3), torch.float16, 0.04)
    maps = []
    for h, w in sizes:
        x = _normal(gen, (1, channels, h, w), torch.float16, 1.0)
        offset = _normal(gen, (1, 18, h, w), torch.float16, 0.5)
        mask = torch.sigmoid(_normal(gen, (1, 9, h, w), torch.float16, 1.0))
        maps.append(mdcn.forward(conv, x, offset, mask, weight)[0].flatten(1).t())
    layer = MapAttention(channels, 8, 8, 64)
    tokens = torch.cat(maps)
    out, saved = layer.forward(tokens, layer.plan(sizes))
    grads = layer.backward(torch.ones_like(out), saved)
    print("maps %s: outputs %s, gradients %s" % (sizes, tuple(out.shape),
                                                 {n: tuple(g.shape) for n, g in grads.items()}))
    decoder = Decoder(channels, 8, 2, 64, batch=2, room=64)
    decoder.prompt(tokens[:12], [5, 7])
    for i in range(4):
        y = decoder.step(tokens[20 + 2 * i:22 + 2 * i])
    print("decoded 4 tokens of 2 sequences: used %s, outputs %s" % (decoder.used.tolist(),
                                                                    tuple(y.shape)))


if __name__ == "__main__":
    main()
