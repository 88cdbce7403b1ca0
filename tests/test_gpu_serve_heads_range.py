"""Head norms where the product of two of value, inverse root and weight is past
the range of 32 bits though the result is not, and where eps counts beside
squares that are past it; within the bounds of serve_heads_util.py."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_heads_util as HU
import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rand(shape, seed, scale):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g).double() * scale).to(torch.bfloat16)


def _check(x, w, eps, what):
    n, _, d = x.shape
    positions = torch.arange(n, dtype=torch.int32)[:, None] * 17
    for rotary_dim in (0, d // 2, d):
        freqs = HU.freqs64(rotary_dim, 10000.0)
        rotation = df11.rotation(rotary_dim) if rotary_dim else None
        out = torch.empty_like(x, device=DEV)
        df11.rotate_heads(x.to(DEV), None, positions[:, 0].contiguous().to(DEV), rotation, out, None, q_weight=w.to(DEV), eps=eps)
        k_out = torch.empty_like(x, device=DEV)
        cache = df11.kv_cache(1, x.shape[1], 16, d)
        df11.kv_append(cache, x.to(DEV), x.to(DEV), positions[:, 0].contiguous().to(DEV), torch.arange(n, device=DEV), rotation, k_weight=w.to(DEV),
                       k_out=k_out, eps=eps)
        torch.cuda.synchronize()
        y, err = HU.heads64(x, positions, freqs, [0] * (rotary_dim // 2), False, 1.0, w, eps)
        U.within(out, y, HU.bound_of(y, err), (what, rotary_dim))
        assert torch.equal(HU.bits(out), HU.bits(k_out)), (what, rotary_dim)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value,weight,eps", [(63, -90, 1e-6), (90, -90, 1e-6), (120, 100, 1e-6), (-49, 100, 2.0 ** -100), (-63, 124, 2.0 ** -100),
                                              (0, 120, 1e-6), (0, -90, 1e-6)])
def test_weights_of_any_size(value, weight, eps, d):
    log(f"norm of values about 2^{value}, weights about 2^{weight}, heads of {d}")
    _check(_rand((5, 3, d), value + 200, 2.0 ** value), _rand((d,), 1, 2.0 ** weight), eps, (value, weight))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value,eps", [(62, 124), (64, 127), (60, 126), (62, 100), (100, 127), (126, 127), (0, 126)])
def test_eps_of_any_size(value, eps, d):
    log(f"norm of values about 2^{value}, eps 2^{eps}, heads of {d}")
    _check(_rand((5, 3, d), value + 300, 2.0 ** value), _rand((d,), 2, 1.0), 2.0 ** eps, (value, eps))


@pytest.mark.parametrize("d", [64, 128])
def test_small_values_beside_a_large_one(d):
    log(f"norm of small values beside a large one, heads of {d}")
    x = _rand((5, 3, d), 7, 2.0 ** -10)
    x[:, :, 9] = 2.0 ** 100
    _check(x, _rand((d,), 3, 2.0 ** 60), 1e-6, d)
