"""attend_token with a sliding window and sinks on the GPU against its
definition in 64 bits (serve_chunk_util.py; a weight is the sum of two BF16
numbers, within 2^-14 of it)."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_chunk_util as CU
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _go(c, q, window, sinks, out=None, **kw):
    out = torch.full_like(q, 7.0) if out is None else out
    df11.attend_token(q, c.cache, c.pages, c.lens, out, window=window, sinks=sinks, **kw)
    torch.cuda.synchronize()
    return out


def _check(c, q, window, sinks, what, **kw):
    got = _go(c, q, window, sinks, **kw)
    import serve_util as U
    U.within(got, *CU.chunk64(q, c.cache, c.table, [1] * len(c.lens_list), c.lens_list, q.shape[2] ** -0.5, True, window, sinks, weights=2.0 ** -14 * 1.01),
             what)
    return got


HEADS = [(4, 1, 128), (6, 6, 64), (20, 1, 64), (8, 2, 128), (40, 2, 128)]
WINDOWS = [(1, 0), (1, 3), (5, 0), (16, 4), (17, 16), (31, 33), (64, 1), (100, 70), (200, 16), (1000, 0), (1500, 100), (5000, 4), (128, 5000)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_windows(window, sinks, int8):
    lens = [1, 0, 16, 17, 64, 199, 333, 1040, 3000]
    for i in range(2):
        h, hk, d = HEADS[(window + 2 * i) % len(HEADS)]
        ps, width = ((16, 300), (64, 0), (256, 20), (32, 0))[(sinks + i) % 4]
        log(f"token in a window of {window}, sinks {sinks}, {h}/{hk} heads of {d}, pages of {ps}, int8 {int8}")
        c = CU.Cached(lens, hk, d, ps, int8, seed=i + window, width=width)
        _check(c, CU.rand((len(lens), h, d), 60 + i), window, sinks, (window, sinks, i))


@pytest.mark.parametrize("int8", [False, True])
def test_every_length_around_the_window(int8):
    """Every offset of the window within a page, a half of a step, and next to the sinks."""
    lens = list(range(1, 140))
    c = CU.Cached(lens, 1, 64, 16, int8, seed=3)
    q = CU.rand((len(lens), 2, 64), 61)
    for window, sinks in ((20, 5), (33, 16), (48, 0), (7, 40)):
        _check(c, q, window, sinks, (window, sinks, int8))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("window,sinks", [(2000, 4), (1500, 700)])
def test_split_windows(window, sinks, int8):
    lens = [9000, 2100, 30, 5555]
    c = CU.Cached(lens, 2, 128, 16, int8, seed=4, width=700)
    q = CU.rand((len(lens), 8, 128), 62)
    need = df11.token_workspace(4, 8, 2, 128, 16, c.pages.shape[1], 0, window, sinks)
    assert need
    ws = torch.full((need // 4,), float("nan"), device=DEV)
    a = _check(c, q, window, sinks, (window, sinks), workspace=ws)
    b = _check(c, q, window, sinks, (window, sinks))
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("int8", [False, True])
def test_keys_out_of_the_window_do_not_reach_the_result(int8):
    lens = [700, 90]
    c = CU.Cached(lens, 1, 64, 16, int8, seed=5)
    q = CU.rand((2, 4, 64), 63)
    clean = _go(c, q, 50, 10)
    k, v, ks, vs = c.cache
    for s, m in enumerate(lens):
        for key in range(10, m - 50):
            page, at = int(c.table[s, key // 16]), key % 16
            for x in ((ks, vs) if int8 else (k, v)):
                x[page, 0, at] = float("nan") if key % 2 else float("inf")
    assert torch.equal(_go(c, q, 50, 10).view(torch.int16), clean.view(torch.int16))
    if not int8:
        page, at = int(c.table[0, 699 // 16]), 699 % 16
        v[page, 0, at, 5] = -float("inf")
        got = _go(c, q, 50, 10)
        assert bool((got[0, :, 5] == -float("inf")).all()) and torch.equal(got[1].view(torch.int16), clean[1].view(torch.int16))


def test_a_window_as_long_as_the_sequence_is_none():
    lens = [300, 1, 77]
    c = CU.Cached(lens, 2, 128, 16, False, seed=6)
    q = CU.rand((3, 4, 128), 64)
    want = _go(c, q, 0, 0)
    for window, sinks in ((10 ** 12, 0), (c.pages.shape[1] * 16, 5), (0, 9)):
        assert torch.equal(_go(c, q, window, sinks), want)
    _check(c, q, 300, 0, "the longest")


def test_wrong_lengths_and_pages():
    lens = [40, 30]
    c = CU.Cached(lens, 2, 64, 16, False, seed=7, poison=False)
    q = CU.rand((2, 4, 64), 65)
    right = _go(c, q, 10, 3)
    c.lens[0] = -1
    got = _go(c, q, 10, 3)
    assert bool((got[0] == 0).all()) and torch.equal(got[1], right[1])
    c.lens[0] = 2 ** 31 - 1
    c.pages[0] = torch.tensor([-1, 2 ** 31 - 1, -7], dtype=torch.int32)
    table = c.table.clone()
    table[0] = c.n_pages - 1
    got = _go(c, q, 10, 3)
    import serve_util as U
    U.within(got, *CU.chunk64(q, c.cache, table, [1, 1], [48, 30], 0.125, True, 10, 3, weights=2.0 ** -14 * 1.01), "the last page")
