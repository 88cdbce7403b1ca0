"""attend_chunk with starts that are out of order or past the rows, with the rows
that are written and those around them; and tiles of 256 rows, which a single
sequence of 2048 rows has in a table of four times its queries, over heads, masks
and values that are not finite."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_chunk_util as CU
import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("longer", [1, 60])
def test_starts_out_of_order(longer, d, int8):
    """A sequence whose rows no other has keeps its results, rows behind the last
    and memory around them are left alone; rows that two sequences have are one's
    or the other's or mixed, which the header leaves open."""
    h, hk, ps = 4, 2, 16
    lens = [40 * longer, 30 * longer, 50 * longer]
    log(f"starts out of order, {lens}, heads of {d}, int8 {int8}")
    c = CU.Cached(lens, hk, d, ps, int8, seed=26)
    q = CU.rand((17, h, d), 67)
    alone, bound = {}, {}
    for s, (a, b) in enumerate([(0, 5), (5, 9), (3, 15)]):
        alone[s], bound[s] = CU.chunk64(q[a:b], c.cache, c.table[s:s + 1], [b - a], lens[s:s + 1], d ** -0.5)

    def go(starts):
        guarded = torch.full((17 + 8, h, d), 7.0, dtype=torch.bfloat16, device=DEV)
        out = guarded[4:21]
        df11.attend_chunk(q[:15], c.cache, c.pages, torch.tensor(starts, dtype=torch.int32, device=DEV), c.lens, out[:15])
        torch.cuda.synchronize()
        assert bool((guarded[:4] == 7).all() and (guarded[19:] == 7).all()), starts
        return out[:15]

    out = go([0, 5, 3, 15])            # the second is passed over, the third begins inside the first
    U.within(out[:3], alone[0][:3], bound[0][:3], "rows of the first alone")
    U.within(out[5:], alone[2][2:], bound[2][2:], "rows of the third alone")
    out = go([-4, 5, 9, 10 ** 6])      # the first begins before the rows, the third ends behind them
    U.within(out[5:9], alone[1], bound[1], "the second")
    assert bool((out[:5] == 7).all() and (out[9:] == 7).all())
    assert bool((go([15, 5, 0, -1]) == 7).all())
    out = go([16, 0, 0, 15])           # the first is passed over, the second empty
    U.within(out, *CU.chunk64(q[:15], c.cache, c.table[2:], [15], lens[2:], d ** -0.5), "the third")


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new,lens,window,sinks", [(600, 600, 0, 0), (517, 1100, 0, 0), (1025, 1025, 100, 70), (700, 3000, 900, 3), (520, 250, 0, 0),
                                                   (512, 9000, 0, 0)])
@pytest.mark.parametrize("h,hk,d,ps", [(8, 2, 128, 16), (8, 2, 64, 64), (20, 1, 64, 32), (5, 1, 128, 128)])
def test_tiles_of_256_rows(h, hk, d, ps, new, lens, window, sinks, int8):
    """Every case in a table of four times its queries at least: 2048 rows in it
    are 256 a tile."""
    log(f"256 rows, {new} of {lens}, window {window} sinks {sinks}, {h}/{hk} heads of {d}, int8 {int8}")
    rows = new + 1
    assert rows * (h // hk) >= 2048
    c = CU.Cached([lens], hk, d, ps, int8, seed=30, width=-(-4 * rows // ps))
    q = CU.rand((rows, h, d), 70)
    size = df11.chunk_workspace(rows, 1, h, hk, d, ps, c.pages.shape[1], window, sinks)
    for causal in (True, False) if not window else (True,):
        out = torch.full_like(q, 7.0)
        df11.attend_chunk(q, c.cache, c.pages, U.starts_of([new]).to(DEV), c.lens, out, causal=causal, window=window, sinks=sinks,
                          workspace=torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        U.within(out[:new], *CU.chunk64(q[:new], c.cache, c.table, [new], [lens], d ** -0.5, causal, window, sinks), (new, lens, causal))
        assert bool((out[new:] == 7.0).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [(600, 700), (520, 4000)])
def test_values_that_are_not_finite_in_tiles_of_256_rows(new, lens, d):
    log(f"not finite, 256 rows, {new} of {lens}, heads of {d}")
    c = CU.Cached([lens], 2, d, 16, False, seed=40, width=-(-4 * new // 16))
    for key, what in ((lens - 150, float("inf")), (lens - 3, float("nan")), (lens - 290, -float("inf"))):
        c.cache.v[int(c.table[0, key // 16]), 0, key % 16, 40] = what
    c.cache.k[int(c.table[0, (lens - 20) // 16]), 1, (lens - 20) % 16, 3] = float("nan")
    q = CU.rand((new, 8, d), 71)
    for window, sinks in ((0, 0), (100, 5)):
        out = torch.full_like(q, 7.0)
        df11.attend_chunk(q, c.cache, c.pages, U.starts_of([new]).to(DEV), c.lens, out, window=window, sinks=sinks)
        torch.cuda.synchronize()
        U.within(out, *CU.chunk64(q, c.cache, c.table, [new], [lens], d ** -0.5, True, window, sinks), (new, lens, window))
