"""The serving calls at the largest sizes that they accept."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("int8", [False, True])
def test_token_over_2_to_the_28_positions(int8):
    """A table of 262,144 pages of 1024: more parts than one dimension of a
    grid holds.  Each quarter of the table is one page again and again, with
    values around a number of its own; the oracle counts how often a position
    is seen."""
    log(f"token over 2^28 positions, int8 {int8}")
    ps, width, h, d = 1024, 1 << 18, 2, 64
    lens = [(1 << 28) - 7, 5]
    g = torch.Generator().manual_seed(9)
    k = torch.randn(4, 1, ps, d, generator=g).to(torch.bfloat16)
    v = (torch.randn(4, 1, ps, d, generator=g) + 8.0 * torch.arange(4)[:, None, None, None]).to(torch.bfloat16)
    ks = vs = None
    if int8:
        (k, ks), (v, vs) = U.quantise32(k), U.quantise32(v)
    cache = df11.KVCache(*(x if x is None else x.to(DEV) for x in (k, v, ks, vs)))
    pages = (torch.arange(width, dtype=torch.int32, device=DEV) >> 16).expand(2, width)
    q = torch.randn(2, h, d, generator=g).to(torch.bfloat16)
    out = torch.empty(2, h, d, dtype=torch.bfloat16, device=DEV)
    df11.attend_token(q.to(DEV), cache, pages, torch.tensor(lens, dtype=torch.int32, device=DEV), out)
    torch.cuda.synchronize()

    kd, vd = (x.double() if s is None else x.double() * s.double()[..., None] for x, s in ((k, ks), (v, vs)))
    kd, vd = kd.reshape(-1, d), vd.reshape(-1, d)
    parts = df11.token_workspace(2, h, 1, d, ps, width) // (2 * h * (d + 2) * 4)
    assert parts > 65536
    for s, seen in enumerate(lens):
        times = torch.zeros(4 * ps, dtype=torch.float64)
        for page in range(4):
            whole = min(max(seen // ps - (page << 16), 0), 1 << 16)
            times[page * ps:(page + 1) * ps] += whole
        rest = seen % ps
        times[(seen // ps >> 16) * ps:][:rest] += 1
        for x in range(h):
            z = kd @ q[s, x].double() * d ** -0.5
            p = torch.where(times > 0, times * torch.exp(z - z.max()), 0.0)
            p = p / p.sum()
            want, a = p @ vd, p @ vd.abs()
            top = float((kd.abs() @ q[s, x].double().abs()).max()) * d ** -0.5
            # the bound of serve_util.py, with sums in 32 bits of a part's keys,
            # and of the parts by four waves
            bound = U.U * want.abs() + a * (U.U * 1.01 + 2 * d * U.E * top + 64 * U.E * (1 + top) + 2 * (ps + parts / 4 + 4) * U.E)
            off = (out[s, x].double().cpu() - want).abs() - bound
            assert float(off.max()) <= 0, (s, x, float(off.max()))
