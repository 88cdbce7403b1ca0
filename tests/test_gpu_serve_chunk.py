"""attend_chunk on the GPU against its definition in 64 bits (serve_chunk_util.py)."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_chunk_util as CU
import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _go(c, q, q_lens, causal=True, window=0, sinks=0, scale=None, out=None, **kw):
    out = torch.full_like(q, 7.0) if out is None else out
    df11.attend_chunk(q, c.cache, c.pages, U.starts_of(q_lens).to(DEV), c.lens, out, causal=causal, window=window, sinks=sinks, scale=scale, **kw)
    torch.cuda.synchronize()
    return out


def _check(c, q, q_lens, what, causal=True, window=0, sinks=0, scale=None, **kw):
    got = _go(c, q, q_lens, causal, window, sinks, scale, **kw)
    n = sum(q_lens)
    want = CU.chunk64(q[:n], c.cache, c.table, q_lens, c.lens_list, q.shape[2] ** -0.5 if scale is None else scale, causal, window, sinks)
    U.within(got[:n], *want, what)
    assert bool((got[n:] == 7.0).all()), what
    return got


# (new tokens, all tokens) of each sequence
MIXES = [
    ([1], [1]),
    ([1, 1, 1], [1, 64, 200]),
    ([5, 1, 70, 1], [5, 17, 70, 333]),
    ([33, 0, 40], [100, 50, 40]),
    ([64], [129]),
    ([7, 3], [4, 0]),                       # more queries than keys; no keys
    ([130, 1, 16], [700, 1000, 16]),
]
HEADS = [(4, 1, 128), (6, 6, 64), (20, 1, 64), (8, 2, 128)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("h,hk,d", HEADS)
def test_mixes(h, hk, d, int8):
    for i, (new, lens) in enumerate(MIXES):
        ps = (16, 64, 128, 32)[i % 4]
        log(f"chunk {new} of {lens}, {h}/{hk} heads of {d}, pages of {ps}, int8 {int8}")
        c = CU.Cached(lens, hk, d, ps, int8, seed=i)
        q = CU.rand((sum(new) + 2, h, d), 50 + i)
        _check(c, q, new, (new, lens))
        _check(c, q, new, (new, lens, "not causal"), causal=False)


WINDOWS = [(1, 0), (1, 3), (16, 4), (63, 0), (64, 64), (65, 1), (100, 70), (200, 16), (5000, 4), (128, 5000)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_windows(window, sinks, int8):
    for i, (new, lens) in enumerate([([40, 1, 150], [40, 700, 900]), ([3, 300], [64, 300]), ([9, 2], [5, 1])]):
        h, hk, d = HEADS[(i + window) % len(HEADS)]
        ps = (16, 64, 32)[i]
        log(f"window {window} sinks {sinks}: {new} of {lens}, {h}/{hk} heads of {d}, int8 {int8}")
        c = CU.Cached(lens, hk, d, ps, int8, seed=i + 7)
        q = CU.rand((sum(new), h, d), 60 + i)
        _check(c, q, new, (new, lens, window, sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new,lens,window,sinks", [([64], [3001], 0, 0), ([20, 1, 77], [3000, 5000, 2477], 0, 0), ([1], [9000], 0, 0),
                                                   ([700, 1], [2000, 4000], 0, 0), ([50, 1], [4000, 3500], 2000, 100), ([900], [900], 600, 4)])
def test_split(new, lens, window, sinks, int8):
    """Sequences whose keys are divided over workgroups, with a workspace of NaN."""
    h, hk, d, ps = (8, 2, 128, 16) if len(new) > 1 else (4, 1, 64, 64)
    log(f"split {new} of {lens}, window {window} sinks {sinks}, int8 {int8}")
    c = CU.Cached(lens, hk, d, ps, int8, seed=20, width=400)
    q = CU.rand((sum(new), h, d), 61)
    need = df11.chunk_workspace(sum(new), len(new), h, hk, d, ps, c.pages.shape[1], window, sinks)
    assert need
    ws = torch.full((need // 4,), float("nan"), device=DEV)
    a = _check(c, q, new, (new, lens), window=window, sinks=sinks, workspace=ws)
    b = _check(c, q, new, (new, lens, "own workspace"), window=window, sinks=sinks)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new,lens,window,sinks", [(600, 600, 0, 0), (517, 1100, 0, 0), (1025, 1025, 100, 70), (700, 3000, 900, 3), (520, 250, 0, 0),
                                                   (512, 9000, 0, 0)])
def test_one_sequence_of_many_rows(new, lens, window, sinks, int8):
    """Tiles of 256 rows, whole and in parts."""
    for i, (h, hk, d, ps) in enumerate([(8, 2, 128, 16), (8, 2, 64, 64), (20, 1, 64, 32), (5, 1, 128, 128)]):
        log(f"one sequence, {new} of {lens}, window {window} sinks {sinks}, {h}/{hk} heads of {d}, int8 {int8}")
        c = CU.Cached([lens], hk, d, ps, int8, seed=30 + i)
        q = CU.rand((new + 1, h, d), 70 + i)
        need = df11.chunk_workspace(new + 1, 1, h, hk, d, ps, c.pages.shape[1], window, sinks)
        ws = torch.full((max(need // 4, 1),), float("nan"), device=DEV)
        _check(c, q, [new], (new, lens, i), window=window, sinks=sinks, workspace=ws)
        if not window:
            _check(c, q, [new], (new, lens, i, "not causal"), causal=False)


@pytest.mark.parametrize("new,lens", [(600, 700), (520, 4000)])
def test_odd_values_in_many_rows(new, lens):
    c = CU.Cached([lens], 2, 128, 16, False, seed=40)
    for key, what in ((lens - 150, float("inf")), (lens - 3, float("nan")), (lens - 290, -float("inf"))):
        c.cache.v[int(c.table[0, key // 16]), 0, key % 16, 40] = what
    c.cache.k[int(c.table[0, (lens - 20) // 16]), 1, (lens - 20) % 16, 3] = float("nan")
    q = CU.rand((new, 8, 128), 71)
    _check(c, q, [new], (new, lens))
    _check(c, q, [new], (new, lens, "window"), window=100, sinks=5)


@pytest.mark.parametrize("n_seqs", [17, 64, 65, 200, 513, 700])
def test_many_sequences(n_seqs):
    log(f"{n_seqs} sequences")
    g = torch.Generator().manual_seed(n_seqs)
    lens = torch.randint(0, 90, (n_seqs,), generator=g).tolist()
    lens[n_seqs // 2] = 2500
    new = [min(m, int(x)) for m, x in zip(lens, torch.randint(0, 40, (n_seqs,), generator=g))]
    new[3] = lens[3] + 2
    c = CU.Cached(lens, 2, 64, 16, False, seed=21)
    q = CU.rand((sum(new) + 1, 4, 64), 62)
    _check(c, q, new, n_seqs)
    _check(c, q, new, (n_seqs, "window"), window=20, sinks=3)


def test_strides_and_results_in_place():
    new, lens = [40, 3], [90, 33]
    c = CU.Cached(lens, 2, 128, 16, False, seed=22)
    rows = CU.rand((sum(new), 12, 128 + 8), 63)
    q = rows[:, 2:10, :128]
    kept = rows.clone()
    want = CU.chunk64(q, c.cache, c.table, new, lens, 128 ** -0.5)
    _go(c, q, new, out=q)
    U.within(q, *want, "in place")
    rows[:, 2:10, :128] = kept[:, 2:10, :128]
    assert torch.equal(rows, kept)
    heads_first = CU.rand((8, sum(new), 128), 64).transpose(0, 1)
    out = torch.empty(8, sum(new), 128, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    _go(c, heads_first, new, out=out)
    U.within(out, *CU.chunk64(heads_first, c.cache, c.table, new, lens, 128 ** -0.5), "heads first")


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("window", [0, 30])
def test_odd_values_reach_only_rows_that_see_them(window, int8):
    log(f"odd values, window {window}, int8 {int8}")
    new, lens = [150, 5], [180, 75]
    for split in (False, True):
        width = 2000 if split else 0
        c = CU.Cached(lens, 2, 64, 16, int8, seed=23, width=width)
        k, v, ks, vs = c.cache
        for s, key, what in ((0, 100, "v+"), (0, 130, "v-"), (0, 160, "vn"), (0, 0, "v+"), (1, 72, "kn"), (0, 177, "kn")):
            page, at = int(c.table[s, key // 16]), key % 16
            if int8:
                (ks if what == "kn" else vs)[page, 0, at] = float("nan")     # (an infinite row reads back as NaN)
            elif what == "kn":
                k[page, 1, at, 3] = float("nan")
            else:
                v[page, 1, at, 7:9] = {"v+": float("inf"), "v-": -float("inf"), "vn": float("nan")}[what]
        q = CU.rand((sum(new), 4, 64), 65)
        _check(c, q, new, (window, int8, split), window=window, sinks=2 if window else 0)


def test_large_values_and_scales():
    new, lens = [20, 1], [400, 1500]
    for d in (64, 128):
        c = CU.Cached(lens, 1, d, 16, False, seed=24)
        c.cache.v.mul_(2.0 ** 120)
        q = CU.rand((sum(new), 4, d), 66, 3.0)
        _check(c, q, new, d)
        c = CU.Cached(lens, 1, d, 16, False, seed=25)
        _check(c, q, new, (d, "sharp"), scale=3.0)
        _check(c, q, new, (d, "flat"), scale=1e-6)


def test_wrong_indexes_stay_inside():
    """Lengths past the table, below zero, pages outside the cache, starts out
    of order: no row of others is hit, and sequences that are right are right."""
    ps, hk, d, h = 16, 2, 64, 4
    lens = [40, 30, 50]
    c = CU.Cached(lens, hk, d, ps, False, seed=26, poison=False)
    new = [5, 4, 6]
    q = CU.rand((15, h, d), 67)
    right = _go(c, q, new)
    c.lens[0] = -3
    got = _go(c, q, new)
    assert bool((got[:5] == 0).all()) and torch.equal(got[5:], right[5:])
    c.lens[0] = 10 ** 9                          # as long as the table
    c.pages[0, :] = torch.tensor([2 ** 31 - 1, -1, 3, 0], dtype=torch.int32)[:c.pages.shape[1]]
    got = _go(c, q, new)
    table = c.table.clone()
    table[0] = torch.tensor([c.n_pages - 1, c.n_pages - 1, 3, 0], dtype=torch.int32)[:c.pages.shape[1]]
    want = CU.chunk64(q, c.cache, table, new, [ps * table.shape[1], 30, 50], d ** -0.5)
    U.within(got, *want, "as long as the table")
    c.lens[0] = 40
    out = torch.full_like(q, 7.0)
    starts = torch.tensor([0, 5, 3, 15], dtype=torch.int32, device=DEV)        # the second is passed over
    df11.attend_chunk(q, c.cache, c.pages, starts, c.lens, out)
    starts = torch.tensor([-4, 5, 9, 10 ** 6], dtype=torch.int32, device=DEV)
    out2 = torch.full_like(q, 7.0)
    df11.attend_chunk(q, c.cache, c.pages, starts, c.lens, out2)
    torch.cuda.synchronize()
    assert torch.equal(out2[5:9], right[5:9]) and bool((out2[:5] == 7).all() and (out2[9:] == 7).all())


@pytest.mark.parametrize("int8", [False, True])
def test_pages_past_32_bits(int8):
    """Byte offsets past 2^32: the last pages of a large cache."""
    log(f"chunk past 2^32 bytes, int8 {int8}")
    pages, hk, d, ps = (1 << 14) + 3, 2 if not int8 else 3, 128, 1024
    cache = df11.kv_cache(pages, hk, ps, d, int8=int8)
    assert cache.k.numel() * cache.k.element_size() > 1 << 32
    lens, new = [1500, 40], [30, 1]
    small = CU.Cached(lens, hk, d, ps, int8, seed=27, poison=False)
    at = torch.tensor([pages - 1 - i for i in range(small.n_pages)], dtype=torch.int32)
    for big, x in zip(cache, small.cache):
        if x is not None:
            big[at.long().to(DEV)] = x
    c = CU.Cached(lens, hk, d, ps, int8, seed=27, poison=False)
    q = CU.rand((sum(new), 2 * hk, d), 68)
    want = CU.chunk64(q, small.cache, small.table, new, lens, d ** -0.5)
    c.cache, c.pages = cache, at[small.table.long()].to(DEV)
    U.within(_go(c, q, new), *want, "far pages")


def test_nothing_to_do():
    c = CU.Cached([5], 1, 64, 16, False, seed=28)
    q = CU.rand((3, 2, 64), 69)
    assert bool((_go(c, q, [0]) == 7).all())
    _go(c, q[:0], [0])
    none = CU.Cached([5], 1, 64, 16, False, seed=28)
    none.lens, none.pages = none.lens[:0], none.pages[:0]
    assert bool((_go(none, q, []) == 7).all())
