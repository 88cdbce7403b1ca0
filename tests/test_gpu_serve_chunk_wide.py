"""attend_chunk on single sequences of 2048 rows and more whose table is wide
(tiles of 256 rows), with and without a prefix, and on either side of the rules
that choose tiles and parts."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_chunk_util as CU
import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(new, total, h, hk, d, ps, int8, causal=True, window=0, sinks=0, positions=0, poison=True):
    log(f"wide {new} of {total} heads {h}/{hk} head_dim {d} page {ps} int8 {int8} causal {causal} window {window} sinks {sinks} positions {positions}")
    c = CU.Cached([total], hk, d, ps, int8, seed=new + total, width=-(-max(positions, total, 1) // ps), poison=poison)
    q = CU.rand((new, h, d), 5)
    out = torch.full_like(q, 7.0)
    size = df11.chunk_workspace(new, 1, h, hk, d, ps, c.pages.shape[1], window, sinks)
    work = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device=DEV)      # (NaN)
    df11.attend_chunk(q, c.cache, c.pages, U.starts_of([new]).to(DEV), c.lens, out, causal=causal, window=window, sinks=sinks, workspace=work)
    torch.cuda.synchronize()
    U.within(out, *CU.chunk64(q, c.cache, c.table, [new], [total], d ** -0.5, causal, window, sinks), (new, total))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,total,h,hk", [(600, 600, 8, 2), (600, 601, 8, 2), (513, 1500, 8, 2), (300, 3333, 16, 2), (300, 250, 16, 2), (300, 0, 16, 2),
                                            (2100, 2100, 2, 2), (110, 5000, 20, 1), (1, 300, 2048, 1)])
def test_wide_tables(new, total, h, hk, d, int8):
    run(new, total, h, hk, d, 16, int8, positions=4 * new + total)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("causal,window,sinks", [(False, 0, 0), (True, 1, 0), (True, 100, 4), (True, 1000, 70), (True, 64, 200), (True, 5000, 3)])
@pytest.mark.parametrize("new,total", [(600, 600), (520, 2600)])
def test_masks(new, total, causal, window, sinks, int8):
    run(new, total, 8, 2, 128, 32, int8, causal, window, sinks, positions=8192)


@pytest.mark.parametrize("positions", [0, 4 * 512 - 16, 4 * 512, 1 << 16])
@pytest.mark.parametrize("new", [511, 512])
def test_either_side_of_the_rules(new, positions):
    """2048 rows, tables of four times the queries; many kv heads, whose parts
    are few."""
    run(new, 700, 4, 1, 64, 16, False, positions=positions)
    run(new, 520, 128, 32, 64, 16, True, positions=positions)


@pytest.mark.parametrize("new,total,h,hk", [(400, 4100, 8, 2), (97, 6400, 8, 2), (130, 3000, 64, 16), (33, 9000, 4, 1)])
def test_parts_of_short_chunks(new, total, h, hk):
    """Parts that are a few more than run at a time, and tiles that are."""
    run(new, total, h, hk, 128, 64, False)
    run(new, total, h, hk, 64, 64, True)


def test_rows_of_16384():
    run(4100, 4100, 4, 1, 64, 64, False)
    run(1030, 1030, 16, 1, 128, 64, True)


def test_values_that_are_not_finite_in_wide_tables():
    """Infinite values at keys that only some rows of a tile of 256 see."""
    c = CU.Cached([700], 2, 128, 16, False, seed=8, width=256)
    for key, x in ((650, float("inf")), (690, float("nan")), (10, float("-inf"))):
        c.cache.v[int(c.table[0, key // 16]), 1, key % 16, 3] = x
    q = CU.rand((600, 8, 128), 9)
    out = torch.empty_like(q)
    df11.attend_chunk(q, c.cache, c.pages, U.starts_of([600]).to(DEV), c.lens, out, window=200)
    torch.cuda.synchronize()
    U.within(out, *CU.chunk64(q, c.cache, c.table, [600], [700], 128 ** -0.5, True, 200, 0), "not finite")


def test_a_captured_graph_follows_the_length():
    """The division of the work is the device's: a graph replayed with other
    lengths divides anew."""
    h, hk, d, new, width = 8, 2, 128, 600, 512
    c = CU.Cached([5000], hk, d, 16, False, seed=4, width=width, poison=False)
    q = CU.rand((new, h, d), 6)
    out = torch.empty_like(q)
    starts = U.starts_of([new]).to(DEV)
    work = torch.empty(df11.chunk_workspace(new, 1, h, hk, d, 16, width), dtype=torch.uint8, device=DEV)
    go = lambda: df11.attend_chunk(q, c.cache, c.pages, starts, c.lens, out, workspace=work)  # noqa: E731
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for n in (5000, 600, 1000, 0, 300, 3001, 5000):
        c.lens.fill_(n)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        U.within(out, *CU.chunk64(q, c.cache, c.table, [new], [n], d ** -0.5), n)
        first = out.clone()
        go()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new,lens,h,hk,d", [([200, 130, 64], [9000, 7000, 5000], 8, 2, 128), ([300, 1, 100, 0], [6100, 6000, 2000, 3000], 8, 1, 64),
                                             ([150] * 8, [2500 - 250 * i for i in range(8)], 8, 2, 64), ([90] * 9, [3100 - 300 * i for i in range(9)], 8, 2, 128),
                                             ([1000, 2], [12000, 12000], 4, 4, 128)])
def test_several_long_sequences(new, lens, h, hk, d, int8):
    """Parts of unequal sequences, up to eight of which are evened out."""
    log(f"several {new} of {lens} heads {h}/{hk} head_dim {d} int8 {int8}")
    c = CU.Cached(lens, hk, d, 64, int8, seed=sum(lens))
    q = CU.rand((sum(new), h, d), 5)
    size = df11.chunk_workspace(len(q), len(new), h, hk, d, 64, c.pages.shape[1])
    memory = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    want, bound = CU.chunk64(q, c.cache, c.table, new, lens, d ** -0.5)
    for _ in range(2):
        out = torch.full_like(q, 7.0)
        df11.attend_chunk(q, c.cache, c.pages, U.starts_of(new).to(DEV), c.lens, out, workspace=memory[:size])
        torch.cuda.synchronize()
        U.within(out, want, bound, new)
        assert bool((memory[size:] == 0xFF).all())
