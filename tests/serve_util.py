"""Oracles of the serving operators (test-side only): the definitions in
include/df11.h on the CPU in 64 bits, and how far BF16 products in 32-bit
accumulators may be from them.

Bound of an attention output, element by element (u = 2^-8 is the largest
relative rounding error of BF16, e = 2^-24 that of 32 bits, A = sum p_j |v_j| /
sum p_j, S = the largest sum of |scale q_d k_d| over a row's keys):
  * the result is rounded to BF16 once: u |o|;
  * weights are rounded to BF16 at most once: u A;
  * a score is a sum of head_dim products in 32 bits, off by at most head_dim e
    S, so that a weight is off by that share, and the sum of weights by as
    much: 2 head_dim e S A; scaling, exponential and the running maximum's
    corrections add a few roundings each: 64 e (1 + S) A;
  * sums over n keys in 32 bits: 2 n e A.
Quantised codes and values read back are compared for equality with the same
operations in 32 bits, and with the definition in 64."""
import math

import torch

U, E = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -100


def attend64(q, k, v, limits, scale):
    """(out, bound) of rows q [n, d] over k, v [m, d] (64 bits, CPU); row i
    sees the first limits[i] keys.  Masked values do not count."""
    n, d = q.shape
    out, bound = torch.zeros(n, d, dtype=torch.float64), torch.zeros(n, d, dtype=torch.float64)
    for i in range(n):
        m = int(limits[i])
        if m <= 0:
            continue
        s = (k[:m] @ q[i]) * scale
        big = s.max()
        if big == -math.inf:
            continue
        p = torch.exp(s - big)
        p = p / p.sum()
        out[i] = p @ v[:m]
        a = p @ v[:m].abs()
        top = ((k[:m].abs() @ q[i].abs()) * scale).max()
        bound[i] = U * out[i].abs() + a * (U * 1.01 + 2 * d * E * top + 64 * E * (1 + top) + 2 * m * E)
    return out, bound


def prompt64(q, k, v, q_lens, k_lens, causal, scale):
    q, k, v = (x.double().cpu() for x in (q, k, v))
    h, hk = q.shape[1], k.shape[1]
    out, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    a = b = 0
    for n, m in zip(q_lens, k_lens):
        limits = [min(max(i + 1 + m - n, 0), m) if causal else m for i in range(n)]
        for x in range(h):
            g = x // (h // hk)
            out[a:a + n, x], bound[a:a + n, x] = attend64(q[a:a + n, x], k[b:b + m, g], v[b:b + m, g], limits, scale)
        a, b = a + n, b + m
    return out, bound


def gathered(store, scale, table, n):
    """The first n tokens' values of one sequence, [n, kv_heads, head_dim] in 64 bits."""
    ps = store.shape[2]
    pages = table[:-(-n // ps)].long()
    x = store[pages].double()
    if scale is not None:
        x = x * scale[pages].double()[..., None]
    return x.transpose(1, 2).flatten(0, 1)[:n]


def token64(q, cache, pages, lens, scale):
    q = q.double().cpu()
    k, v, ks, vs = (None if x is None else x.cpu() for x in cache)
    pages = pages.cpu()
    b, h, d = q.shape
    hk = k.shape[1]
    out, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for s in range(b):
        n = int(lens[s])
        if n == 0:
            continue
        kd, vd = gathered(k, ks, pages[s], n), gathered(v, vs, pages[s], n)
        for x in range(h):
            g = x // (h // hk)
            o, e = attend64(q[s, x][None], kd[:, g], vd[:, g], [n], scale)
            out[s, x], bound[s, x] = o[0], e[0]
    return out, bound


def within(got, out, bound, what):
    """Every element of got (BF16) within the bound of out; NaN or infinite
    where out is."""
    got = got.double().cpu()
    odd = ~torch.isfinite(out)
    assert torch.equal(torch.isnan(got), torch.isnan(out)), (what, "NaN in other places")
    assert torch.equal(got[odd & ~torch.isnan(out)], out[odd & ~torch.isnan(out)]), (what, "infinities in other places")
    off = ((got - out).abs() - bound)[~odd]
    assert off.numel() == 0 or float(off.max()) <= 1e-30, (what, float(off.max()), int((off > 0).sum()), off.numel())


def quantise32(x):
    """(codes, scales) of BF16 rows, by the definition's operations in 32 bits."""
    x = x.float().cpu()
    a = x.abs().amax(-1).clamp_min(TINY)
    inv = torch.full_like(a, 127.0) / a
    codes = torch.round(x * inv[..., None])
    return torch.where(torch.isnan(codes), torch.zeros_like(codes), codes).to(torch.int8), a / 127.0


def make_tables(lens, page_size, seed, extra=2, width=0):
    """Page tables over shuffled pages (CPU int32), and the number of pages."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // page_size) for n in lens]
    n_pages = sum(need) + extra
    order = torch.randperm(n_pages, generator=gen).to(torch.int32)
    width = max(width, 1, *need)
    t = torch.zeros(len(lens), width, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, n_pages


def starts_of(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int64).cumsum(0).to(torch.int32)
