"""attend_chunk in 8 bits over few keys: weights of two BF16 operands, within
2^-14 of each weight (rows that see up to 512 keys, causal or not, windows,
split or not), where longer tiles are held to weights rounded once."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_chunk_util as CU
import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
TWO = 2.0 ** -14 * 1.01


@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (False, 0, 0), (True, 3, 4), (True, 100, 17)])
@pytest.mark.parametrize("new,lens,h,hk,d", [([2], [452], 12, 4, 128), ([60, 2, 0, 17], [60, 500, 30, 512], 8, 2, 64), ([200, 151], [512, 151], 20, 1, 128),
                                             ([5] * 70, [5 + 7 * (i % 60) for i in range(70)], 4, 2, 128)])
def test_few_keys_in_8_bits(new, lens, h, hk, d, causal, window, sinks):
    log(f"few keys {new} of {lens} heads {h}/{hk} head_dim {d} causal {causal} window {window} sinks {sinks}")
    c = CU.Cached(lens, hk, d, 16, True, seed=sum(lens))
    q = CU.rand((sum(new), h, d), 7, 1.5)
    out = torch.full_like(q, 7.0)
    df11.attend_chunk(q, c.cache, c.pages, U.starts_of(new).to(DEV), c.lens, out, causal=causal, window=window, sinks=sinks)
    torch.cuda.synchronize()
    U.within(out, *CU.chunk64(q, c.cache, c.table, new, lens, d ** -0.5, causal, window, sinks, weights=TWO), (causal, window))


def test_the_bound_tells_them_apart():
    """Weights rounded once, which a tile of more than 512 keys has, lie outside
    the narrower bound."""
    c = CU.Cached([700], 2, 128, 16, True, seed=3)
    q = CU.rand((64, 8, 128), 8, 1.5)
    out = torch.empty_like(q)
    df11.attend_chunk(q, c.cache, c.pages, U.starts_of([64]).to(DEV), c.lens, out, causal=False)
    torch.cuda.synchronize()
    U.within(out, *CU.chunk64(q, c.cache, c.table, [64], [700], 128 ** -0.5, False), "rounded once")
    want, bound = CU.chunk64(q, c.cache, c.table, [64], [700], 128 ** -0.5, False, weights=TWO)
    assert bool(((out.double().cpu() - want).abs() > bound).any())
