"""Layers of whole numbers whose decode step has one right answer, bit for bit.

Every weight is code x scale with a scale of 1 or 2 per group, x is a whole number, and
each row of W1, W3 and W2 has a few values that are not 0, one in each part of the row:
  gate  two columns of x hold 8 and W1 holds 2 there: G = 32 + three terms of at most
        2 * 2 * 1, so 20 <= G <= 44, where exp(-G) < 2^-25 and silu(G) = G in float32;
  up    three terms of at most 3 * 2 * 1: |U| <= 18, so |G U| <= 792;
  h     G U is exact in float32 and has one rounding to bf16;
  y     a slot's sum has six terms of at most 8 * 2 * 792, and k <= 16 slots weigh 1/2 to 2:
        below 2^22, in units of 1/2.
The 4-bit products sum 24 h and (24 + code) h over a group of at most 128: below
128 * 55 * 792 < 2^23.  So every float32 sum is exact in whatever order it is taken, and y is
the sum in 64 bits, rounded once to bf16.
"""
import numpy as np
import torch

import synth


def bf(a):
    """a rounded to bf16, as float32."""
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(np.asarray(a, np.float32)))


def pack(codes):
    """Bytes [..][cols / 2] of codes [..][cols] (int8, -8 to 7) on their device: code k + i of a word of
    eight, plus 8, at bit 4 (i / 2 + 4 (i % 2))."""
    c = (codes.view(*codes.shape[:-1], -1, 8) + 8).to(torch.int32)
    word = torch.zeros_like(c[..., 0])
    for i in range(8):
        word |= c[..., i] << (4 * (i // 2 + 4 * (i % 2)))
    return word.view(torch.uint8)


def _places(rng, rows, cols, n):
    """n different columns of each row, one in each n-th of it."""
    edge = np.arange(n + 1) * cols // n
    return np.stack([rng.integers(edge[i], edge[i + 1], rows) for i in range(n)], axis=1)


def _nonzero(rng, lo, hi, shape):
    v = rng.integers(lo, hi, shape)  # lo .. hi - 1, 0 left out
    return np.where(v >= 0, v + 1, v)


class Layer:
    """x, a given routing, and sparse weights {name: (columns, codes)} with scales by group (bf16 layers: of 64)."""

    def __init__(self, T, d, f, E, k, e0, NL, group, seed):
        rng = np.random.default_rng(seed)
        self.T, self.d, self.f, self.E, self.k, self.e0, self.NL, self.group = T, d, f, E, k, e0, NL, group
        g = group or 64
        self.x = rng.choice([-1.0, 1.0], (T, d)).astype(np.float32)
        carry = np.array([d // 3, d - 2])
        self.x[:, carry] = 8
        # two picks in three go to a few experts, so that some have many tokens and others one or none
        few = rng.permutation(E)[:max(1, E // 8)]
        self.idx = np.where(rng.random((T, k)) < 2 / 3, rng.choice(few, (T, k)), rng.integers(0, E, (T, k))).astype(np.int32)
        self.w = rng.choice([0.5, 1.0, 2.0], (T, k)).astype(np.float32)
        self.at, self.code, self.scale = {}, {}, {}
        for name, rows, cols, n, lo, hi in (("w1", f, d, 3, -2, 2), ("w3", f, d, 3, -3, 3), ("w2", d, f, 6, -8, 7)):
            at = _places(rng, NL * rows, cols, n)
            code = _nonzero(rng, lo, hi, at.shape)
            scale = rng.choice([1.0, 2.0], (NL * rows, -(-cols // g))).astype(np.float32)
            if name != "w2":
                code[np.isin(at, carry)] = 0
            if name == "w1":
                at = np.concatenate([at, np.broadcast_to(carry, (NL * rows, 2))], axis=1)
                code = np.concatenate([code, 2 // np.take_along_axis(scale, np.broadcast_to(carry // g, (NL * rows, 2)), 1).astype(int)], axis=1)
            self.at[name], self.code[name], self.scale[name] = at, code, scale

    def values(self, name):
        """The values at the columns at[name], [NL][rows][n]."""
        v = self.code[name] * np.take_along_axis(self.scale[name], self.at[name] // (self.group or 64), 1)
        return v.reshape(self.NL, -1, v.shape[1])

    def weights(self, name, device):
        """bf16 weights [NL][rows][cols], or 4-bit bytes and scales."""
        rows, cols = (self.d, self.f) if name == "w2" else (self.f, self.d)
        at = torch.from_numpy(np.ascontiguousarray(self.at[name])).to(device)
        # (added: a column named twice has a code of 0 once)
        if self.group:
            q = torch.zeros(self.NL * rows, cols, dtype=torch.int8, device=device)
            q.scatter_add_(1, at, torch.from_numpy(self.code[name].astype(np.int8)).to(device))
            return (pack(q).view(self.NL, rows, cols // 2),
                    torch.from_numpy(self.scale[name]).to(device).view(self.NL, rows, -1))
        v = torch.zeros(self.NL * rows, cols, dtype=torch.bfloat16, device=device)
        val = self.values(name).reshape(self.NL * rows, -1)
        return v.scatter_add_(1, at, torch.from_numpy(val).to(device).bfloat16()).view(self.NL, rows, cols)

    def y(self, skip=None, without=None, scales=None):
        """y [T][d] (float32 holding bf16 values).  For planted mistakes: skip = (name, lo, hi) leaves columns
        lo .. hi - 1 of a matrix out, without leaves one local expert out, scales = (name, group) takes the
        scales of one group twice over."""
        val = {n: self.values(n).astype(np.float64) for n in self.at}
        at = {n: self.at[n].reshape(self.NL, -1, self.at[n].shape[1]) for n in self.at}
        if skip:
            val[skip[0]] = np.where((at[skip[0]] >= skip[1]) & (at[skip[0]] < skip[2]), 0, val[skip[0]])
        if scales:
            val[scales[0]] = np.where(at[scales[0]] // (self.group or 64) == scales[1], 2, 1) * val[scales[0]]
        x = self.x.astype(np.float64)
        y = np.zeros((self.T, self.d))
        for e in range(self.NL):
            t, j = np.nonzero(self.idx - self.e0 == e)
            if len(t) == 0 or e == without:
                continue
            G = (x[t][:, at["w1"][e]] * val["w1"][e]).sum(axis=2)
            U = (x[t][:, at["w3"][e]] * val["w3"][e]).sum(axis=2)
            assert skip or scales or (G.min() >= 20 and G.max() <= 44 and np.abs(U).max() <= 18)
            h = bf(G * U).astype(np.float64)
            out = (h[:, at["w2"][e]] * val["w2"][e]).sum(axis=2)
            np.add.at(y, t, self.w[t, j][:, None].astype(np.float64) * out)
        assert np.abs(y).max() < 2 ** 22 and (y * 2 == np.rint(y * 2)).all()
        return bf(y)


# T, d, f, E, k, expert_begin, local experts, and the form that 256 CUs run: bf16 (tokens, tokens a block, rows of a
# gate/up stage, channels of d), 4 bits
FORMS = [
    ((1, 640, 320, 16, 4, 0, 16), (2, 2, 16, 8), (2, 2, 32, 8)),
    ((1, 4160, 64, 8, 2, 0, 8), (2, 2, 16, 24), (2, 2, 32, 24)),
    ((2, 640, 320, 16, 4, 4, 12), (2, 2, 16, 8), (2, 2, 32, 8)),
    ((2, 4160, 192, 8, 3, 0, 8), (2, 2, 16, 24), (2, 2, 32, 24)),
    ((3, 832, 448, 24, 3, 0, 24), (16, 16, 16, 8), (16, 4, 16, 8)),
    ((9, 640, 192, 24, 3, 2, 20), (16, 16, 16, 8), (16, 4, 16, 8)),
    ((16, 576, 128, 8, 8, 0, 8), (16, 16, 16, 8), (16, 4, 16, 8)),
    ((12, 4160, 64, 16, 4, 0, 16), (16, 16, 16, 24), (16, 4, 16, 24)),
    ((8, 640, 320, 64, 8, 0, 64), (16, 16, 16, 8), (16, 4, 32, 8)),
    ((16, 2048, 1024, 32, 8, 0, 32), (16, 16, 16, 8), (16, 4, 32, 8)),
    ((16, 4160, 256, 64, 4, 0, 64), (16, 16, 16, 24), (16, 4, 32, 24)),
    ((17, 640, 320, 24, 3, 0, 24), (64, 12, 16, 8), (64, 8, 32, 8)),
    ((64, 576, 192, 40, 5, 5, 30), (64, 12, 16, 8), (64, 8, 32, 8)),
    ((33, 4160, 320, 8, 2, 0, 8), (64, 12, 16, 24), (64, 8, 32, 24)),
    ((64, 4160, 64, 16, 8, 0, 16), (64, 12, 16, 24), (64, 8, 32, 24)),
]


# Of a layer with random weights: h and y are rounded to bf16, by at most 2^-8 of each value.  h's roundings come to a
# column of y through W2, whose signs do not depend on them: at most 2^-8 of a token's rms; y's own are at most 2^-8 of
# the block's rms, which is below 1.5 of the token's for 64 random columns.  Float32 sums add less than 2^-14.
BLOCK_TOL = 2.0 ** -8 * (1 + 1.5) + 2.0 ** -14


def worst_block(got, want):
    """The largest rms of got - want over 64 columns of a token, in the token's rms (NaN counts as infinite)."""
    err = np.asarray(got, np.float64) - want
    rms = np.sqrt((want ** 2).mean(axis=1))
    worst = 0.0
    for lo in range(0, want.shape[1], 64):
        b = np.sqrt((err[:, lo:lo + 64] ** 2).mean(axis=1)) / rms
        worst = max(worst, float(np.where(np.isfinite(b), b, np.inf).max()))
    return worst
