"""Oracle of rotate_heads and kv_append (test-side only): the definition in
include/df11.h on the CPU in 64 bits, and how far results in 32 bits, rounded
to BF16 once, may be from it.

Bound of an element that comes from the pair (a, b) by a c - b s (u = 2^-8 is
the largest relative rounding error of BF16, e = 2^-24 that of 32 bits):
  * the phase is exact; its float is within e of it, at most half a turn: an
    angle off by pi e, and the sine unit is within 2^-22 of the sine (found for
    2^25 phases over the whole turn and next to 0): 2^-22 + pi e < 2^-21 of
    |a| + |b|; products, their sum and the factor round four times: 4 e (|a| + |b|);
  * the norm: a sum of head_dim squares in 32 bits is off by at most head_dim e
    of itself, its square root by half of that; mean, root, weight and product
    round six times: (head_dim / 2 + 6) e of each element;
  * the result is rounded to BF16 once: u of it (2^-134 below the normal numbers)."""
import math

import torch

U, E = 2.0 ** -8, 2.0 ** -24


def freqs64(rotary_dim, base):
    return [base ** (-2 * i / rotary_dim) for i in range(rotary_dim // 2)]


def heads64(x, positions, freqs, axes, neighbours, factor=1.0, weight=None, eps=1e-6):
    """(y, err): x [n, heads, d] normed and rotated in 64 bits, and how far it
    may be from that before it is rounded.  freqs: radians a position;
    positions [n, axes]."""
    x = x.double().cpu()
    n, _, d = x.shape
    err = torch.zeros_like(x)
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double().cpu()
        err = x.abs() * ((d / 2 + 6) * E)
    y, pairs = x.clone(), len(freqs)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + pairs)
        # (position * f in 64 bits is off by 2^-53 of itself: turns modulo 1 by whole numbers)
        turns = round(math.fmod(f / (2 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64
        at = [(int(p) * turns % 2 ** 64) / 2.0 ** 64 for p in positions[:, axes[i]].tolist()]
        t = torch.tensor(at, dtype=torch.float64)[:, None] * (2 * math.pi)
        c, s = torch.cos(t), torch.sin(t)
        y[..., a], y[..., b] = factor * (x[..., a] * c - x[..., b] * s), factor * (x[..., b] * c + x[..., a] * s)
        more = abs(factor) * ((x[..., a].abs() + x[..., b].abs()) * (2.0 ** -21 + 4 * E) + err[..., a] + err[..., b])
        err[..., a] = err[..., b] = more
    return y, err


def bound_of(y, err):
    return U * y.abs() + (1 + U) * err + 2.0 ** -134


def bits(x):
    return x.contiguous().view(torch.int16)
