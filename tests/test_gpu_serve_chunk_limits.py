"""attend_chunk, windows and heads at the ends of what the calls allow: 2^28
positions a sequence, many kv heads, broadcast and strided inputs, scales that
are infinite."""
import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_chunk_util as CU
import serve_heads_util as HU
import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new,window,sinks", [(1, 0, 0), (2, 0, 0), (2, (1 << 28) - 1000, 700), (1, (1 << 28) - 1000, 700)])
def test_2_to_the_28_positions(new, window, sinks, int8):
    """A table of 262,144 pages of 1024.  Each quarter of it is one page again
    and again, with values around a number of its own; the oracle counts how
    often each row is seen by each query."""
    log(f"chunk of {new} over 2^28 positions, window {window}, int8 {int8}")
    ps, width, h, d = 1024, 1 << 18, 2, 64
    n = (1 << 28) - 7
    g = torch.Generator().manual_seed(9)
    k = torch.randn(4, 1, ps, d, generator=g).to(torch.bfloat16)
    v = (torch.randn(4, 1, ps, d, generator=g) + 8.0 * torch.arange(4)[:, None, None, None]).to(torch.bfloat16)
    ks = vs = None
    if int8:
        (k, ks), (v, vs) = U.quantise32(k), U.quantise32(v)
    cache = df11.KVCache(*(x if x is None else x.to(DEV) for x in (k, v, ks, vs)))
    pages = (torch.arange(width, dtype=torch.int32, device=DEV) >> 16).expand(1, width)
    q = torch.randn(new, h, d, generator=g).to(torch.bfloat16)
    out = torch.empty(new, h, d, dtype=torch.bfloat16, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, new], dtype=torch.int32, device=DEV)
    df11.attend_chunk(q.to(DEV), cache, pages, starts, lens, out, window=window, sinks=sinks)
    results = [out]
    if new == 1 and window:
        results.append(torch.empty_like(out))
        df11.attend_token(q.to(DEV), cache, pages, lens, results[1], window=window, sinks=sinks)
    torch.cuda.synchronize()

    kd, vd = (x.double() if s is None else x.double() * s.double()[..., None] for x, s in ((k, ks), (v, vs)))
    kd, vd = kd.reshape(-1, d), vd.reshape(-1, d)

    def times(end):
        """How often each of the 4 x 1024 rows lies below position `end`."""
        t = torch.zeros(4 * ps, dtype=torch.float64)
        for page in range(4):
            t[page * ps:(page + 1) * ps] += min(max(end // ps - (page << 16), 0), 1 << 16)
        t[(end // ps >> 16) * ps:][:end % ps] += 1
        return t

    for i in range(new):
        end = n - new + i + 1
        seen = times(end) - (times(end - window) - times(sinks) if window else 0)
        for x in range(h):
            z = kd @ q[i, x].double() * d ** -0.5
            p = torch.where(seen > 0, seen * torch.exp(z - z.max()), 0.0)
            p = p / p.sum()
            want, a = p @ vd, p @ vd.abs()
            top = float((kd.abs() @ q[i, x].double().abs()).max()) * d ** -0.5
            # the bound of serve_util.py, with sums in 32 bits of a part's keys (at
            # most 2^28 / 256 where 512 parts are asked for and rounded, eight of
            # which join at once) of one lane: a quarter of them, or a half
            # (attend_token's weights are rounded less; its sums are shorter)
            bound = U.U * want.abs() + a * (U.U * 1.01 + 2 * d * U.E * top + 64 * U.E * (1 + top) + 2 * ((1 << 28) / 256 / 2 + 512) * U.E)
            for got in results:
                off = (got[i, x].double().cpu() - want).abs() - bound
                assert float(off.max()) <= 0, (i, x, float(off.max()))


def test_many_kv_heads():
    """More kv heads than parts could be given."""
    h, hk, d = 600, 300, 64
    lens, new = [700, 40], [3, 40]
    c = CU.Cached(lens, hk, d, 16, False, seed=1, width=100)
    q = CU.rand((sum(new), h, d), 2)
    out = torch.empty_like(q)
    df11.attend_chunk(q, c.cache, c.pages, U.starts_of(new).to(DEV), c.lens, out)
    torch.cuda.synchronize()
    U.within(out, *CU.chunk64(q, c.cache, c.table, new, lens, d ** -0.5), "many kv heads")
    assert df11.chunk_workspace(43, 2, 1000, 500, d, 16, 1 << 12) == 0


def test_broadcast_and_strided_inputs():
    """Rows that share their memory, positions of one column of several."""
    n, h, hk, d = 40, 4, 2, 64
    one = CU.rand((1, 1, d), 3)
    q, k = one.expand(n, h, d), one.expand(n, hk, d)
    table = torch.arange(4 * n, dtype=torch.int32, device=DEV).view(n, 4)
    r = df11.rotation(d)
    qo, ko = (torch.empty(n, x, d, dtype=torch.bfloat16, device=DEV) for x in (h, hk))
    df11.rotate_heads(q, k, table[:, 2], r, qo, ko)
    torch.cuda.synchronize()
    for got, x in ((qo, q), (ko, k)):
        y, err = HU.heads64(x, table[:, 2:3].cpu(), HU.freqs64(d, 10000.0), [0] * (d // 2), False)
        U.within(got, y, HU.bound_of(y, err), "strided positions")
    # the same position for all tokens
    df11.rotate_heads(q, None, table[5:6, 1].expand(n), r, qo, None)
    torch.cuda.synchronize()
    y, err = HU.heads64(q, table[5:6, 1:2].cpu().expand(n, 1), HU.freqs64(d, 10000.0), [0] * (d // 2), False)
    U.within(qo, y, HU.bound_of(y, err), "one position")
    lens = [90]
    c = CU.Cached(lens, hk, d, 16, False, seed=4)
    out = torch.empty(n, h, d, dtype=torch.bfloat16, device=DEV)
    df11.attend_chunk(q, c.cache, c.pages, U.starts_of([n]).to(DEV), c.lens, out)
    torch.cuda.synchronize()
    U.within(out, *CU.chunk64(q, c.cache, c.table, [n], lens, d ** -0.5), "broadcast queries")


@pytest.mark.parametrize("window", [0, 25])
def test_scales_that_are_infinite(window):
    """A row that held an infinity has codes 0 and a scale of infinity: NaN for
    those who see it, nothing for others."""
    new, lens = [60, 1], [100, 300]
    c = CU.Cached(lens, 2, 64, 16, True, seed=5)
    for s, key, which in ((0, 70, 2), (0, 90, 3), (1, 100, 3), (1, 299 - 24, 2)):
        page, at = int(c.table[s, key // 16]), key % 16
        c.cache[which - 2][page, 1, at] = 0
        c.cache[which][page, 1, at] = float("inf")
    q = CU.rand((sum(new), 4, 64), 6)
    out = torch.empty_like(q)
    df11.attend_chunk(q, c.cache, c.pages, U.starts_of(new).to(DEV), c.lens, out, window=window)
    torch.cuda.synchronize()
    want, bound = CU.chunk64(q, c.cache, c.table, new, lens, 0.125, True, window, 0)
    assert torch.equal(torch.isnan(out).cpu(), torch.isnan(want)) and bool(torch.isnan(want).any()) and not bool(torch.isnan(want).all())
    U.within(out, want, bound, window)


@pytest.mark.parametrize("n_seqs,width", [(9, 32), (131, 32), (9, 4096)])
def test_starts_that_do_not_ascend_stay_inside(n_seqs, width):
    """Sequences over the same rows: more tiles than the rows could hold.  The
    results are not defined; the memory around workspace and output is."""
    h, hk, d, n, guard = 8, 2, 64, 100, 1 << 20
    lens = [width * 16] * n_seqs
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(8, hk, 16, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    pages = torch.randint(0, 8, (n_seqs, width), generator=g, dtype=torch.int32).to(DEV)
    starts = torch.tensor([0, n] * ((n_seqs + 1) // 2), dtype=torch.int32, device=DEV)
    size = df11.chunk_workspace(n, n_seqs, h, hk, d, 16, width)
    assert size > 0
    memory = torch.full((size + guard,), 0x5A, dtype=torch.uint8, device=DEV)
    out = torch.full((n + 64, h, d), 7.0, dtype=torch.bfloat16, device=DEV)
    for _ in range(2):
        df11.attend_chunk(CU.rand((n, h, d), 4), df11.KVCache(k, v), pages, starts, torch.tensor(lens, dtype=torch.int32, device=DEV), out[:n], workspace=memory[:size])
    torch.cuda.synchronize()
    assert bool((memory[size:] == 0x5A).all()) and bool((out[n:] == 7.0).all())
