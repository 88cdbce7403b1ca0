"""attend_token within the bound of two-operand weights (serve_precision.py):
results that are small beside what they sum, few keys with most of the weight,
and the plain random rows of the other tests."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_precision as P
import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,ps,h,hk,d", [([2, 16, 33, 300, 1000], 16, 8, 2, 128), ([2, 16, 33, 300, 1000], 32, 8, 2, 64),
                                            ([5000, 300, 0, 33], 16, 8, 2, 128), ([5000, 1000], 64, 20, 1, 64),
                                            ([1, 15, 17, 31, 32, 127, 129], 16, 3, 3, 64)])
def test_token_weights(lens, ps, h, hk, d, int8):
    log(f"token weights {lens} page {ps} heads {h}/{hk} head_dim {d} int8 {int8}")
    t, n_pages = U.make_tables(lens, ps, 3)
    g = torch.Generator().manual_seed(11)
    shape = (n_pages, hk, ps, d)
    k, v = (torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2))
    for cancel in (True, False):
        if cancel:
            for s, n in enumerate(lens):        # each sequence's values in nearly cancelling pairs
                pages = t[s, :-(-n // ps)].long()
                rows = P.balanced(v[pages].transpose(1, 2).flatten(0, 1))
                v[pages] = rows.unflatten(0, (len(pages), ps)).transpose(1, 2)
        else:
            v = torch.randn(shape, generator=g).to(torch.bfloat16)
        scales, stored = [None, None], [k, v]
        if int8:
            (ck, ks), (cv, vs) = U.quantise32(k), U.quantise32(v)
            scales, stored = [ks, vs], [ck, cv]
        cache = df11.KVCache(*(x if x is None else x.to(DEV) for x in (*stored, *scales)))
        q = (4.0 if cancel else 1.5) * torch.randn(len(lens), h, d, generator=g)
        q = q.to(torch.bfloat16).to(DEV)
        out = torch.empty_like(q)
        df11.attend_token(q, cache, t.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), out)
        U.within(out, *P.token64(q, cache, t, lens, d ** -0.5), (lens, int8, cancel))
