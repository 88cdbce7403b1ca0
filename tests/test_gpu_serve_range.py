"""Finite inputs of any size give finite results: values up to the largest
BF16 number, seen by many keys, over sums that are kept as the keys come.

attend_prompt rounds a weight to BF16 once, by at most 2^-8 of it, and the last
1/256 below 2^128 rounds to infinity, so its values end 2^-6 below the largest
number; attend_token's weights are within 2^-14, and its values end with it."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
MOST = torch.finfo(torch.bfloat16).max


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


def _large(shape, seed, most=MOST):
    """Values between half and the whole of `most`, of one sign in even columns
    and of both in odd ones."""
    g = torch.Generator().manual_seed(seed)
    x = (0.5 + 0.5 * torch.rand(shape, generator=g, dtype=torch.float64)) * most
    x[..., 0] = most
    sign = torch.where(torch.rand(shape, generator=g) < 0.5, -1.0, 1.0)
    sign[..., ::2] = 1
    return (x * sign).to(torch.bfloat16).to(DEV)


def _rising(k, q):
    """Keys whose scores rise by little from one to the next, so that the
    running maximum lags behind."""
    n = k.shape[0]
    k[:] = (q[-1, :1].float() / q[-1, :1].float().norm() * torch.linspace(0, 4, n, device=DEV)[:, None, None]).to(torch.bfloat16)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,m", [(1, 2), (70, 70), (200, 333), (40, 3000)])
def test_prompt_largest_values(n, m, d, causal):
    log(f"prompt, largest values: {n} on {m}, head_dim {d}, causal {causal}")
    h = 2
    s, t = (U.starts_of([x]).to(DEV) for x in (n, m))
    v = _large((m, 1, d), 3, MOST * (1 - 2.0 ** -6))
    for rising in (False, True):
        q, k = _rand((n, h, d), 1), _rand((m, 1, d), 2)
        if rising:
            _rising(k, q)
        out = torch.empty_like(q)
        df11.attend_prompt(q, k, v, s, t, out, causal=causal)
        U.within(out, *U.prompt64(q, k, v, [n], [m], causal, d ** -0.5), (n, m, rising))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,ps,d", [([1, 2, 40, 300], 16, 128), ([900, 31], 32, 64), ([6000, 40], 16, 128)])
def test_token_largest_values(lens, ps, d, int8):
    log(f"token, largest values: {lens}, head_dim {d}, int8 {int8}")
    h = 4
    t, n_pages = U.make_tables(lens, ps, 5)
    q = _rand((len(lens), h, d), 7)
    for rising in (False, True):
        k, v = _rand((n_pages, 1, ps, d), 8), _large((n_pages, 1, ps, d), 9)
        if rising:
            at = t[0].long()
            rows = torch.empty(len(at) * ps, 1, d, dtype=torch.bfloat16, device=DEV)
            _rising(rows, q[:1])
            k[at.to(DEV)] = rows.view(len(at), ps, 1, d).transpose(1, 2)
        ks = vs = None
        if int8:
            (k, ks), (v, vs) = ((x.to(DEV) for x in U.quantise32(x)) for x in (k, v))
        cache = df11.KVCache(k, v, ks, vs)
        out = torch.empty_like(q)
        df11.attend_token(q, cache, t.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), out)
        U.within(out, *U.token64(q, cache, t, lens, d ** -0.5), (lens, rising))


@pytest.mark.parametrize("int8", [False, True])
def test_largest_values_are_written_and_read(int8):
    log(f"largest values through the cache, int8 {int8}")
    n, d = 20, 128
    k, v = _large((n, 1, d), 11), -_large((n, 1, d), 12)
    cache = df11.kv_cache(2, 1, 16, d, int8=int8)
    df11.kv_write(cache, k, v, torch.arange(n, device=DEV))
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    df11.kv_read(cache, torch.arange(2, dtype=torch.int32, device=DEV)[None], U.starts_of([n]).to(DEV), ko, vo)
    for got, rows in ((ko, k), (vo, v)):
        want = rows
        if int8:
            codes, scales = U.quantise32(rows)
            want = (codes.float() * scales[..., None]).to(torch.bfloat16).to(DEV)
        assert torch.isfinite(got.float()).all() and torch.equal(got, want)
