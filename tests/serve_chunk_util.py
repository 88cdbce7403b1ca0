"""Oracle of attend_chunk and of windows (test-side only): the definition in
include/df11.h on the CPU in 64 bits, with the bounds of serve_util.py."""
import math

import torch

import serve_util as U


def seen64(n, m, causal, window, sinks):
    """[n, m]: whether query i of n, at position m - n + i, sees key j."""
    at, key = torch.arange(m - n, m)[:, None], torch.arange(m)[None, :]
    if not causal:
        return torch.ones(n, m, dtype=torch.bool)
    seen = key <= at
    if window:
        seen &= (key > at - window) | (key < sinks)
    return seen


def attend64(q, k, v, seen, scale, weights=U.U * 1.01):
    """(out, bound) of rows q [n, d] over k, v [m, d], in 64 bits; `weights`:
    what rounding a weight costs, relative."""
    n, d = q.shape
    m = k.shape[0]
    z = torch.where(seen, (q @ k.T) * scale, -math.inf)
    big = z.amax(-1, keepdim=True) if m else torch.full((n, 1), -math.inf, dtype=torch.float64)
    p = torch.exp(z - torch.where(torch.isinf(big) & (big < 0), 0.0, big))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    odd = ~torch.isfinite(v)
    finite = torch.where(odd, 0.0, v)
    out, a = p @ finite, p @ finite.abs()
    if bool(odd.any()):
        with_key = ((p > 0) | torch.isnan(p)).double()
        up, down, nan = ((with_key @ x.double()) > 0 for x in (v == math.inf, v == -math.inf, torch.isnan(v)))
        out = torch.where(up, math.inf, out)
        out = torch.where(down, -math.inf, out)
        out = torch.where(nan | (up & down), math.nan, out)
    size = torch.where(seen, (q.abs() @ k.abs().T) * scale, 0.0)
    top = size.amax(-1, keepdim=True) if m else torch.zeros(n, 1, dtype=torch.float64)
    keys = seen.sum(-1, keepdim=True)
    bound = U.U * out.abs() + a * (weights + 2 * d * U.E * top + 64 * U.E * (1 + top) + 2 * keys * U.E)
    return out, bound


def chunk64(q, cache, pages, q_lens, lens, scale, causal=True, window=0, sinks=0, weights=U.U * 1.01):
    q = q.double().cpu()
    k, v, ks, vs = (None if x is None else x.cpu() for x in cache)
    pages = pages.cpu()
    h, hk = q.shape[1], k.shape[1]
    out, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    a = 0
    for s, (n, m) in enumerate(zip(q_lens, lens)):
        if n and m:
            kd, vd = U.gathered(k, ks, pages[s], m), U.gathered(v, vs, pages[s], m)
            seen = seen64(n, m, causal, window, sinks)
            for x in range(h):
                g = x // (h // hk)
                out[a:a + n, x], bound[a:a + n, x] = attend64(q[a:a + n, x], kd[:, g], vd[:, g], seen, scale, weights)
        a += n
    return out, bound


class Cached:
    """A cache of random keys and values on the GPU with shuffled pages, in
    words or 8 bits; unused rows hold NaN (scales of NaN) where `poison`."""

    def __init__(self, lens, hk, d, ps, int8, seed, width=0, poison=True, device="cuda"):
        import lossless_bf16_weight_amd as df11
        t, n_pages = U.make_tables(lens, ps, seed, width=width)
        g = torch.Generator().manual_seed(seed)
        k, v = (torch.randn(n_pages, hk, ps, d, generator=g).to(torch.bfloat16) for _ in range(2))
        used = torch.zeros(n_pages, ps, dtype=torch.bool)
        for s, m in enumerate(lens):
            at = torch.arange(m)
            used[t[s, at // ps].long(), at % ps] = True
        scales = [None, None]
        if int8:
            (k, ks), (v, vs) = U.quantise32(k), U.quantise32(v)
            scales = [ks, vs]
        if poison:
            hide = ~used[:, None, :].expand(n_pages, hk, ps)
            for x in (scales if int8 else (k, v)):
                x[hide] = float("nan")
        self.lens_list, self.n_pages = list(lens), n_pages
        self.cache = df11.KVCache(*(None if x is None else x.to(device) for x in (k, v, *scales)))
        self.table = t
        past = t.clone()
        for s, m in enumerate(lens):      # (entries past a length are not read)
            past[s, -(-m // ps):] = -5 if s % 2 else 2 ** 31 - 1
        self.pages = past.to(device)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=device)


def rand(shape, seed, scale=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(device)
