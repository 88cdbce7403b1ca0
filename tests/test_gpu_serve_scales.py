"""Attention over a cache in 8 bits whose scales are of either sign, or infinite (a
code times its scale is the value, whatever that is), with scores so far apart that
weights are 0 in 32 bits: against the definition in 64 bits (serve_chunk_util.py)."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_chunk_util as CU
import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _signed(lens, hk, d, ps, seed, width=0):
    c = CU.Cached(lens, hk, d, ps, True, seed=seed, width=width)
    g = torch.Generator().manual_seed(seed + 1)
    for x in c.cache[2:]:
        x.mul_(torch.randint(0, 2, x.shape, generator=g).to(DEV) * 2 - 1)
    return c


@pytest.mark.parametrize("scale", [None, 3.0])
@pytest.mark.parametrize("h,hk,d,ps", [(4, 1, 128, 16), (8, 2, 64, 64), (20, 1, 64, 16), (20, 1, 128, 32)])
def test_tokens(h, hk, d, ps, scale):
    lens = [1, 40, 300, 1024, 2500]
    log(f"signed scales, tokens over {lens}, {h}/{hk} heads of {d}, scale {scale}")
    c = _signed(lens, hk, d, ps, 1)
    q = CU.rand((len(lens), h, d), 2, 3.0)
    s = d ** -0.5 if scale is None else scale
    for window, sinks in ((0, 0), (100, 3)):
        want = CU.chunk64(q, c.cache, c.table, [1] * len(lens), lens, s, True, window, sinks)
        out = torch.full_like(q, 7.0)
        df11.attend_token(q, c.cache, c.pages, c.lens, out, scale=scale, window=window, sinks=sinks)
        U.within(out, *want, ("token", window))
        out = torch.full_like(q, 7.0)
        df11.attend_chunk(q, c.cache, c.pages, U.starts_of([1] * len(lens)).to(DEV), c.lens, out, scale=scale, window=window, sinks=sinks)
        U.within(out, *want, ("chunk", window))


@pytest.mark.parametrize("scale", [None, 3.0])
@pytest.mark.parametrize("new,lens", [([40, 1, 70], [40, 333, 500]), ([130, 20], [2000, 700]), ([600], [900])])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks(new, lens, d, scale):
    log(f"signed scales, chunk {new} of {lens}, heads of {d}, scale {scale}")
    c = _signed(lens, 2, d, 16, 3, width=160)
    q = CU.rand((sum(new), 8, d), 4, 3.0)
    s = d ** -0.5 if scale is None else scale
    for window, sinks in ((0, 0), (100, 3)):
        out = torch.full_like(q, 7.0)
        df11.attend_chunk(q, c.cache, c.pages, U.starts_of(new).to(DEV), c.lens, out, scale=scale, window=window, sinks=sinks)
        U.within(out, *CU.chunk64(q, c.cache, c.table, new, lens, s, True, window, sinks), window)


def test_results_stay_with_scales_that_are_not_negative():
    """Turning a key's codes and its scale to the other sign changes no bit."""
    lens = [60, 700]
    c = CU.Cached(lens, 2, 128, 16, True, seed=5, poison=False)
    q = CU.rand((2, 8, 128), 6, 3.0)
    k, v, ks, vs = c.cache
    turned = df11.KVCache(-k, -v, -ks, -vs)
    starts = U.starts_of([1, 1]).to(DEV)
    for go in (lambda cache, out: df11.attend_token(q, cache, c.pages, c.lens, out, scale=2.0),
               lambda cache, out: df11.attend_chunk(q, cache, c.pages, starts, c.lens, out, scale=2.0)):
        a, b = torch.empty_like(q), torch.empty_like(q)
        go(c.cache, a)
        go(turned, b)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_scales_of_values(sign, d):
    """Codes other than 0 times an infinite scale are infinities, for the rows that
    see them."""
    new, lens = [40, 1], [300, 2500]
    log(f"scales of {sign} infinity, heads of {d}")
    c = _signed(lens, 2, d, 16, 7)
    for s, key in ((0, 280), (1, 2000)):
        page, at = int(c.table[s, key // 16]), key % 16
        c.cache.v[page, 1, at] = torch.arange(1, d + 1, dtype=torch.int8, device=DEV)
        c.cache.v_scale[page, 1, at] = sign * float("inf")
    q = CU.rand((sum(new), 8, d), 8)
    for window in (0, 100):
        want, bound = CU.chunk64(q, c.cache, c.table, new, lens, d ** -0.5, True, window, 0)
        out = torch.full_like(q, 7.0)
        df11.attend_chunk(q, c.cache, c.pages, U.starts_of(new).to(DEV), c.lens, out, window=window)
        U.within(out, want, bound, ("chunk", window))
        assert bool(torch.isinf(want).any()) and not bool(torch.isinf(want).all())
        out = torch.full_like(q[-1:], 7.0)
        df11.attend_token(q[-1:], c.cache, c.pages[1:], c.lens[1:], out, window=window)
        U.within(out, want[-1:], bound[-1:], ("token", window))
