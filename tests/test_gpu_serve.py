"""GPU parity of the key-value cache and the attention operators against the
definitions in 64 bits (serve_util.py): lengths of zero and one, sizes on both
sides of every tile, rows that see no key, pages that end inside a tile, grouped
heads, strides, stray infinities and NaN where no row looks, page numbers and
lengths out of range, long offsets, streams and graphs."""
import math

import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


def _guarded(shape):
    """A BF16 output between two guard rows, filled with 0x5A5A."""
    buf = torch.full((shape[0] + 2, *shape[1:]), 0x5A5A, dtype=torch.int16, device=DEV)
    return buf, buf[1:-1].view(torch.bfloat16)


def _guards_hold(buf):
    assert bool((buf[0] == 0x5A5A).all()) and bool((buf[-1] == 0x5A5A).all()), "wrote outside the output"


# ------------------------------------------------------------------- prompts

PROMPTS = [
    # q_lens, k_lens (None: the same), heads, kv_heads, head_dim, causal
    ([1], None, 1, 1, 128, True),
    ([2], [1], 2, 1, 128, True),
    ([64], None, 4, 1, 128, True),
    ([64], None, 4, 1, 64, True),
    ([31, 33, 1, 0, 63, 65], None, 4, 2, 128, True),
    ([127, 128, 129], None, 3, 1, 64, True),
    ([127, 1, 128, 129, 0, 191, 193], None, 2, 2, 128, False),
    ([5, 200, 17], [130, 64, 17], 8, 2, 128, True),          # behind a prefix, and more queries than keys
    ([140, 3], [0, 70], 2, 1, 64, True),                     # no keys at all
    ([140, 3], [0, 70], 2, 1, 128, False),
    ([1] * 70 + [40] + [2] * 60, None, 2, 1, 64, True),      # more sequences than a wave has lanes
    ([257], [300], 5, 5, 128, False),
    ([300], None, 20, 1, 64, True),
]


def _prompt_inputs(q_lens, k_lens, h, hk, d, seed):
    n, m = sum(q_lens), sum(k_lens)
    return _rand((n, h, d), seed, 1.5), _rand((m, hk, d), seed + 1, 1.5), _rand((m, hk, d), seed + 2)


@pytest.mark.parametrize("case", PROMPTS)
def test_prompt(case):
    q_lens, k_lens, h, hk, d, causal = case
    k_lens = q_lens if k_lens is None else k_lens
    log(f"prompt {case}")
    q, k, v = _prompt_inputs(q_lens, k_lens, h, hk, d, 1)
    buf, out = _guarded(q.shape)
    df11.attend_prompt(q, k, v, U.starts_of(q_lens).to(DEV), U.starts_of(k_lens).to(DEV), out, causal=causal)
    torch.cuda.synchronize()
    _guards_hold(buf)
    U.within(out, *U.prompt64(q, k, v, q_lens, k_lens, causal, d ** -0.5), case)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 40, 63, 64, 65, 130])
def test_prompt_counts_of_sequences(n):
    """The ways to find a work item's sequence; a third of the sequences empty,
    whole and ragged tiles, with keys in one part and in several."""
    log(f"prompt of {n} sequences")
    h, hk, d = 6, 2, 64
    q_lens = [(0, 43, 1, 128, 0, 86, 17, 0, 129)[(5 * i + n) % 9] for i in range(n)]
    for extra in (0, 1200):
        k_lens = [m + extra * (i % 13 == 3) for i, m in enumerate(q_lens)]
        q, k, v = _prompt_inputs(q_lens, k_lens, h, hk, d, n)
        buf, out = _guarded(q.shape)
        df11.attend_prompt(q, k, v, U.starts_of(q_lens).to(DEV), U.starts_of(k_lens).to(DEV), out)
        torch.cuda.synchronize()
        _guards_hold(buf)
        U.within(out, *U.prompt64(q, k, v, q_lens, k_lens, True, d ** -0.5), (n, extra))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,m", [(1, 4096), (40, 3000), (130, 2049), (700, 1600), (900, 650)])
def test_prompt_split_over_keys(n, m, d):
    """Few rows over many keys: the keys are split and the parts joined, the
    second sequence too short for all parts."""
    log(f"prompt split {n} over {m}, head_dim {d}")
    q_lens, k_lens, h, hk = [n, 7], [m, 600], 4, 2
    q, k, v = _prompt_inputs(q_lens, k_lens, h, hk, d, 5)
    need = df11.prompt_workspace(sum(q_lens), sum(k_lens), 2, h, hk, d)
    assert need > 0
    want = U.prompt64(q, k, v, q_lens, k_lens, True, 0.05)
    a, b = U.starts_of(q_lens).to(DEV), U.starts_of(k_lens).to(DEV)
    outs = []
    for ws in (None, torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)):    # (NaN where nothing is written)
        buf, out = _guarded(q.shape)
        df11.attend_prompt(q, k, v, a, b, out, scale=0.05, workspace=ws)
        torch.cuda.synchronize()
        _guards_hold(buf)
        U.within(out, *want, (n, m, d))
        outs.append(out.view(torch.int16).cpu())
    assert torch.equal(*outs)
    with pytest.raises(df11.DF11Error):
        df11.attend_prompt(q, k, v, a, b, out, workspace=torch.empty(need - 16, dtype=torch.uint8, device=DEV))


def test_prompt_strides_and_in_place():
    """Queries, keys and values as parts of one projection's output, heads
    before rows, one key row for every position, and the result over q."""
    log("prompt strides")
    lens, h, hk, d = [77, 150], 4, 2, 128
    n = sum(lens)
    s = U.starts_of(lens).to(DEV)
    fused = _rand((n, h + 2 * hk, d), 11)
    q, k, v = fused[:, :h], fused[:, h:h + hk], fused[:, h + hk:]
    want = U.prompt64(q, k, v, lens, lens, True, d ** -0.5)
    out = torch.empty(n, h, d, dtype=torch.bfloat16, device=DEV)
    df11.attend_prompt(q, k, v, s, s, out)
    U.within(out, *want, "fused")
    by_head = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    out_h = torch.empty(h, n, d, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    df11.attend_prompt(*by_head, s, s, out_h)
    assert torch.equal(out_h, out)
    same = q.clone()
    df11.attend_prompt(same, k, v, s, s, same)
    assert torch.equal(same, out)
    one_v = v[:1].expand(n, hk, d)
    df11.attend_prompt(q, k, one_v, s, s, out)
    U.within(out, *U.prompt64(q, k, one_v, lens, lens, True, d ** -0.5), "broadcast values")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("split", [False, True])
def test_prompt_other_sequences_do_not_matter(bad, split):
    """A sequence of infinities or NaN next to others leaves them as they are,
    its own rows aside."""
    log(f"prompt beside {bad}, split {split}")
    q_lens = [30, 50, 20]
    k_lens = [700, 650, 720] if split else q_lens
    h, hk, d = 2, 1, 128
    q, k, v = _prompt_inputs(q_lens, k_lens, h, hk, d, 21)
    a, b = U.starts_of(q_lens).to(DEV), U.starts_of(k_lens).to(DEV)
    good, out = torch.empty_like(q), torch.empty_like(q)
    df11.attend_prompt(q, k, v, a, b, good)
    at = U.starts_of(k_lens)
    k[at[1]:at[2]] = bad
    v[at[1]:at[2]] = bad
    df11.attend_prompt(q, k, v, a, b, out)
    for lo, hi in ((0, 30), (80, 100)):
        assert torch.equal(out[lo:hi], good[lo:hi])
    assert not bool(torch.isfinite(out[30:80].float()).any())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("split", [False, True])
def test_prompt_masked_values_do_not_matter(split, d):
    """Causal rows before a key whose value (or key) is infinite or NaN are
    what they are without it, in the same step of keys too; the rows that see
    it get what the definition gives."""
    log(f"prompt masked infinities, split {split}, head_dim {d}")
    n, m, h, hk = (70, 1200, 4, 1) if split else (200, 200, 3, 1)
    q, k, v = _prompt_inputs([n], [m], h, hk, d, 25)
    a, b = U.starts_of([n]).to(DEV), U.starts_of([m]).to(DEV)
    assert (df11.prompt_workspace(n, m, 1, h, hk, d) > 0) == split
    out = torch.empty_like(q)
    first = m - n
    for at, value in ((first + 40, math.inf), (first + 41, -math.inf), (first + 62, math.nan), (m - 1, math.nan), (m - 3, math.inf)):
        bad = v.clone()
        bad[at, 0, d // 2] = value
        bad[at, 0, 3] = -value
        df11.attend_prompt(q, k, bad, a, b, out)
        U.within(out, *U.prompt64(q, k, bad, [n], [m], True, d ** -0.5), ("value", at, value))
        assert torch.isfinite(out[:at - first].float()).all() and not torch.isfinite(out[at - first:, :, 3].float()).any()
    bad = v.clone()       # both infinities at one place: NaN from the second on
    bad[first + 20, 0, 5], bad[first + 50, 0, 5] = math.inf, -math.inf
    df11.attend_prompt(q, k, bad, a, b, out)
    U.within(out, *U.prompt64(q, k, bad, [n], [m], True, d ** -0.5), "both")
    bad = k.clone()
    bad[first + 45] = math.nan
    df11.attend_prompt(q, bad, v, a, b, out)
    U.within(out[:45], *(x[:45] for x in U.prompt64(q, k, v, [n], [m], True, d ** -0.5)), "key")
    assert torch.isnan(out[45:].float()).all()


def test_prompt_starts_out_of_order():
    """Sequences whose starts are not in order within the rows are passed
    over: their rows keep what they held."""
    log("prompt starts out of order")
    h, d = 2, 64
    q, k, v = _rand((100, h, d), 31), _rand((100, h, d), 32), _rand((100, h, d), 33)
    ok = torch.tensor([0, 40, 100], dtype=torch.int32, device=DEV)
    for starts in ([0, 40, 101], [0, 40, 2 ** 31 - 1], [0, 40, 30], [0, 40, -5]):
        bad = torch.tensor(starts, dtype=torch.int32, device=DEV)
        for a, b in ((bad, bad), (ok, bad)):
            out = torch.full((100, h, d), 9.0, dtype=torch.bfloat16, device=DEV)
            df11.attend_prompt(q, k, v, a, b, out, causal=False)
            want = U.prompt64(q[:40], k[:40], v[:40], [40], [40], False, d ** -0.5)
            U.within(out[:40], *want, starts)
            assert bool((out[40:] == 9.0).all()), starts


def test_prompt_extreme_scores():
    """Scores of plus and minus 1e4 and of minus infinity: one key takes all,
    rows whose scores are all minus infinity are zero."""
    log("prompt extreme scores")
    n, d = 70, 64
    q, k, v = _rand((n, 1, d), 41, 30.0), _rand((n, 1, d), 42, 30.0), _rand((n, 1, d), 43)
    s = U.starts_of([n]).to(DEV)
    out = torch.empty_like(q)
    df11.attend_prompt(q, k, v, s, s, out, scale=1.0)
    U.within(out, *U.prompt64(q, k, v, [n], [n], True, 1.0), "large")
    q[:] = 1
    k[:] = -math.inf
    df11.attend_prompt(q, k, v, s, s, out)
    assert bool((out == 0).all())


# -------------------------------------------------------------------- tokens

def _cache(lens, ps, hk, d, int8, seed, poison=None, width=0):
    """(cache, tables): random cached rows; every position of no sequence holds
    `poison` where one is given."""
    t, n_pages = U.make_tables(lens, ps, seed, width=width)
    k, v = _rand((n_pages, hk, ps, d), seed + 1, 1.5), _rand((n_pages, hk, ps, d), seed + 2)
    ks = vs = None
    if int8:
        (k, ks), (v, vs) = ((x.to(DEV) for x in U.quantise32(x)) for x in (k, v))
    if poison is not None:
        used = torch.zeros(n_pages, ps, dtype=torch.bool)
        for i, n in enumerate(lens):
            for j in range(n):
                used[t[i, j // ps], j % ps] = True
        free = ~used.to(DEV)
        if int8:
            for x in (ks, vs):
                x.masked_fill_(free[:, None, :], poison)
        else:
            for x in (k, v):
                x.masked_fill_(free[:, None, :, None], poison)
    return df11.KVCache(k, v, ks, vs), t.to(DEV)


TOKENS = [
    # lens, page_size, heads, kv_heads, head_dim
    ([1], 16, 1, 1, 128),
    ([0, 1, 15, 16, 17, 31, 32, 33], 16, 4, 1, 128),
    ([0, 1, 15, 16, 17, 31, 32, 33], 16, 4, 1, 64),
    ([127, 128, 129, 255, 257, 511, 513], 32, 8, 2, 128),
    ([700, 0, 3], 64, 5, 5, 64),
    ([300, 299], 128, 20, 1, 128),
    ([1000, 1], 1024, 16, 2, 64),
    ([5000, 4095, 4097, 0], 16, 8, 1, 128),
    ([1023, 384, 0, 1024, 385, 31], 16, 8, 2, 128),            # taken whole by twelve waves
    ([500, 900], 32, 20, 1, 64),
]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("case", TOKENS)
def test_token(case, int8):
    lens, ps, h, hk, d = case
    log(f"token {case} int8 {int8}")
    for poison in (None, math.nan, math.inf):
        cache, pages = _cache(lens, ps, hk, d, int8, 3, poison)
        q = _rand((len(lens), h, d), 7, 1.5)
        buf, out = _guarded(q.shape)
        df11.attend_token(q, cache, pages, torch.tensor(lens, dtype=torch.int32, device=DEV), out)
        torch.cuda.synchronize()
        _guards_hold(buf)
        U.within(out, *U.token64(q, cache, pages, lens, d ** -0.5), (case, int8, poison))


@pytest.mark.parametrize("lens", [[1, 2, 40, 300], [900, 31], [6000, 40]])
def test_token_infinite_values_that_are_seen(lens):
    """Values that are infinite at keys that count: the result is infinite
    there, and NaN where both infinities meet; others stay."""
    log(f"token with infinite values {lens}")
    ps, h, hk, d = 16, 4, 2, 128
    cache, pages = _cache(lens, ps, hk, d, False, 43)
    at = [(j // ps, j % ps) for j in (0, 1, 17, 30)]
    for s, n in enumerate(lens):
        for column, ((page, pos), value) in enumerate(zip(at, (math.inf, -math.inf, math.inf, math.nan))):
            if page * ps + pos < n:
                cache.v[pages[s, page], 0, pos, column] = value
        if n > 30:
            cache.v[pages[s, 0], 1, 2, 64], cache.v[pages[s, 1], 1, 3, 64] = math.inf, -math.inf
    q = _rand((len(lens), h, d), 47, 0.5)
    out = torch.empty_like(q)
    df11.attend_token(q, cache, pages, torch.tensor(lens, dtype=torch.int32, device=DEV), out)
    U.within(out, *U.token64(q, cache, pages, lens, d ** -0.5), lens)


@pytest.mark.parametrize("int8", [False, True])
def test_token_split_and_workspace(int8):
    """A wide table splits the work; short sequences leave most parts empty.
    The workspace starts as NaN."""
    log(f"token split int8 {int8}")
    lens, ps, h, hk, d = [9000, 1, 0, 2500], 16, 8, 2, 128
    cache, pages = _cache(lens, ps, hk, d, int8, 13, width=2000)
    q = _rand((len(lens), h, d), 17)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    need = df11.token_workspace(len(lens), h, hk, d, ps, 2000)
    assert need > 0
    want = U.token64(q, cache, pages, lens, 0.1)
    outs = []
    for ws in (None, torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)):
        buf, out = _guarded(q.shape)
        df11.attend_token(q, cache, pages, ln, out, scale=0.1, workspace=ws)
        torch.cuda.synchronize()
        _guards_hold(buf)
        U.within(out, *want, int8)
        outs.append(out.view(torch.int16).cpu())
    assert torch.equal(*outs)
    with pytest.raises(df11.DF11Error):
        df11.attend_token(q, cache, pages, ln, out, workspace=torch.empty(need - 16, dtype=torch.uint8, device=DEV))


def test_token_strides_and_ranges():
    """q as part of a projection's output, a table that is a part of a wider
    one, the result over q; lengths past the table and page numbers past the
    cache stay inside it."""
    log("token strides")
    lens, ps, h, hk, d = [100, 37], 16, 4, 2, 128
    cache, pages = _cache(lens, ps, hk, d, False, 23)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    fused = _rand((2, h + 2 * hk, d), 29)
    q = fused[:, :h]
    wide = torch.full((2, 40), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
    wide[:, 3:3 + pages.shape[1]] = pages
    part = wide[:, 3:3 + pages.shape[1]]
    want = U.token64(q, cache, pages, lens, d ** -0.5)
    out = torch.empty(2, h, d, dtype=torch.bfloat16, device=DEV)
    df11.attend_token(q, cache, part, ln, out)
    U.within(out, *want, "strided")
    same = q.clone()
    df11.attend_token(same, cache, part, ln, same)
    assert torch.equal(same, out)
    # length past the table: the table's positions count; below zero: none
    df11.attend_token(q, cache, pages, torch.tensor([2 ** 31 - 1, -3], dtype=torch.int32, device=DEV), out)
    full = pages.shape[1] * ps
    U.within(out, *U.token64(q, cache, pages, [full, 0], d ** -0.5), "length")
    # page numbers past the cache, above and below: its last page
    odd = pages.clone()
    odd[0, 1], odd[0, 2], odd[1, 0] = 2 ** 31 - 1, -1, cache.k.shape[0]
    last = odd.clone()
    last[0, 1] = last[0, 2] = last[1, 0] = cache.k.shape[0] - 1
    df11.attend_token(q, cache, odd, ln, out)
    U.within(out, *U.token64(q, cache, last, lens, d ** -0.5), "pages")


@pytest.mark.parametrize("int8", [False, True])
def test_token_nan_in_a_sequence_stays_there(int8):
    log(f"token NaN int8 {int8}")
    lens, ps, h, hk, d = [50, 40], 16, 2, 2, 64
    cache, pages = _cache(lens, ps, hk, d, int8, 33)
    q = _rand((2, h, d), 37)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    good, out = torch.empty_like(q), torch.empty_like(q)
    df11.attend_token(q, cache, pages, ln, good)
    where = cache.v_scale if int8 else cache.v
    where[pages[0, 1].item(), 1, 5] = math.nan          # sequence 0, kv head 1
    df11.attend_token(q, cache, pages, ln, out)
    assert torch.equal(out[1], good[1]) and torch.equal(out[0, 0], good[0, 0])
    assert bool(torch.isnan(out[0, 1]).all())


# --------------------------------------------------------------------- cache

@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,ps,hk,d", [([1], 16, 1, 64), ([5, 0, 16, 17, 100], 16, 3, 128), ([63, 64, 65, 129, 1], 32, 2, 64),
                                          ([300, 200], 256, 8, 128), ([70, 0, 5, 17], 16, 40, 128), ([33, 1], 128, 24, 64)])
def test_write_then_read(lens, ps, hk, d, int8):
    """Codes and scales equal those of the same operations in 32 bits, are
    within half a step of the definition in 64, touch no other slot, and read
    back as the rounded products (words: as the words)."""
    log(f"write and read {lens} page {ps} int8 {int8}")
    n = sum(lens)
    t, n_pages = U.make_tables(lens, ps, 41)
    slots = torch.cat([t[i, torch.arange(m) // ps].long() * ps + torch.arange(m) % ps for i, m in enumerate(lens)])
    fused = _rand((n, 4 * hk, d), 43, 3.0)
    k, v = fused[:, hk:2 * hk], fused[:, 3 * hk:]
    fused[0, hk, :] = 0                                        # a row of zeros
    if n > 2:
        fused[1, hk] = 2.0 ** -120                             # below 2^-100: codes 0
        fused[2, hk, 1:] = 0                                   # one value alone
    cache = df11.kv_cache(n_pages, hk, ps, d, int8=int8)
    for x in cache:
        if x is not None:
            x.fill_(77)
    df11.kv_write(cache, k, v, slots.to(DEV))
    torch.cuda.synchronize()
    want = [torch.full_like(x, 77).cpu() if x is not None else None for x in cache]
    page, at = slots // ps, slots % ps
    for i, rows in enumerate((k, v)):
        if int8:
            codes, scales = U.quantise32(rows)
            want[i][page, :, at], want[2 + i][page, :, at] = codes, scales
            x = rows.double().cpu()
            a = x.abs().amax(-1, keepdim=True).clamp_min(U.TINY)
            assert float((codes.double() - x * 127 / a).abs().max()) <= 0.5 + 127 * 2.0 ** -22
        else:
            want[i][page, :, at] = rows.cpu()
    for x, w in zip(cache, want):
        assert x is None or torch.equal(x.cpu(), w)
    kb, ko = _guarded((n, hk, d))
    vb, vo = _guarded((n, hk, d))
    df11.kv_read(cache, t.to(DEV), U.starts_of(lens).to(DEV), ko, vo)
    torch.cuda.synchronize()
    for buf, got, store, scale in ((kb, ko, want[0], want[2]), (vb, vo, want[1], want[3])):
        _guards_hold(buf)
        values = store[page, :, at].float()
        if int8:
            values = values * scale[page, :, at][..., None]
        assert torch.equal(got.cpu(), values.to(torch.bfloat16))


def test_write_slots_outside_and_not_finite():
    log("write slots outside")
    hk, d, ps, n_pages = 2, 64, 16, 3
    k, v = _rand((6, hk, d), 51), _rand((6, hk, d), 52)
    k[0, 0, 3], k[1, 1, 0], v[2, 0, 63] = math.inf, math.nan, -math.inf
    slots = torch.tensor([0, 47, 5, -1, 48, 2 ** 40], device=DEV)
    for int8 in (False, True):
        cache = df11.kv_cache(n_pages, hk, ps, d, int8=int8)
        df11.kv_write(cache, k, v, slots)
        n = 48
        ko, vo = (torch.empty(n, hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        table = torch.arange(3, dtype=torch.int32, device=DEV)[None]
        df11.kv_read(cache, table, torch.tensor([0, n], dtype=torch.int32, device=DEV), ko, vo)
        written = torch.zeros(n, dtype=torch.bool)
        written[[0, 47, 5]] = True
        assert bool((ko.cpu()[~written] == 0).all()) and bool((vo.cpu()[~written] == 0).all())
        if not int8:
            assert torch.equal(ko[[0, 47, 5]].view(torch.int16), k[:3].view(torch.int16))
        else:
            assert bool(torch.isnan(ko[0, 0]).all()) and bool(torch.isnan(ko[47, 1]).all()) and bool(torch.isnan(vo[5, 0]).all())
            assert bool(torch.isfinite(ko[[0, 47, 5]][[0, 1, 2], [1, 0, 0]].float()).all())


def test_read_ranges():
    """Starts out of order or past the rows leave their sequence out; page
    numbers past the cache read its last page; sequences longer than the table
    end with it."""
    log("read ranges")
    hk, d, ps = 1, 64, 16
    cache, pages = _cache([40, 40], ps, hk, d, False, 61)
    for starts in ([0, 40, 81], [0, 40, 39], [0, 40, -1]):
        ko, vo = (torch.full((80, hk, d), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        df11.kv_read(cache, pages, torch.tensor(starts, dtype=torch.int32, device=DEV), ko, vo)
        assert torch.equal(ko[:40].double().cpu(), U.gathered(cache.k.cpu(), None, pages[0].cpu(), 40))
        assert bool((ko[40:] == 9.0).all()) and bool((vo[40:] == 9.0).all())
    odd = pages.clone()
    odd[0, 0], odd[1, 1] = -7, 2 ** 31 - 1
    last = odd.clone()
    last[0, 0] = last[1, 1] = cache.k.shape[0] - 1
    ko, vo = (torch.full((120, hk, d), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    df11.kv_read(cache, odd, torch.tensor([0, 40, 120], dtype=torch.int32, device=DEV), ko, vo)
    assert torch.equal(vo[:40].double().cpu(), U.gathered(cache.v.cpu(), None, last[0].cpu(), 40))
    assert torch.equal(vo[40:88].double().cpu(), U.gathered(cache.v.cpu(), None, last[1].cpu(), 48))
    assert bool((vo[88:] == 9.0).all())


def test_offsets_past_32_bits():
    """Pages past 2^31 elements and 2^32 bytes of the cache, and query rows
    that far apart."""
    log("long offsets")
    hk, ps, d, n_pages = 8, 16, 128, 140000          # 2.3e9 elements, 4.6 GB each
    cache = df11.KVCache(*(torch.empty(n_pages, hk, ps, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    pages = torch.tensor([[n_pages - 1, 0, n_pages - 2]], dtype=torch.int32, device=DEV)
    n = 40
    k, v = _rand((n, hk, d), 71, 1.5), _rand((n, hk, d), 72)
    at = torch.arange(n, device=DEV)
    df11.kv_write(cache, k, v, pages[0, at // ps].long() * ps + at % ps)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    s = U.starts_of([n]).to(DEV)
    df11.kv_read(cache, pages, s, ko, vo)
    assert torch.equal(ko, k) and torch.equal(vo, v)
    q = _rand((1, 16, d), 73)
    out = torch.empty_like(q)
    df11.attend_token(q, cache, pages, torch.tensor([n], dtype=torch.int32, device=DEV), out)
    want = U.prompt64(q, k, v, [1], [n], True, d ** -0.5)
    U.within(out, *want, "token")
    m, stride = 130, 2 ** 24 - 8                     # key rows 32 MB apart, 4.3 GB in all
    k, v = _rand((m, hk, d), 75, 1.5), _rand((m, hk, d), 76)
    kf, vf = (torch.as_strided(x.view(-1), (m, hk, d), (stride, d, 1)) for x in cache[:2])
    kf.copy_(k)
    vf.copy_(v)
    qs = torch.as_strided(cache.k.view(-1), (m, 1, d), (stride, d, 1), 2 ** 20)
    qs.copy_(_rand((m, 1, d), 74))
    os = torch.as_strided(cache.v.view(-1), (m, 1, d), (stride, d, 1), 2 ** 20)
    s = U.starts_of([m]).to(DEV)
    df11.attend_prompt(qs, kf[:, :1], vf[:, :1], s, s, os)
    U.within(os, *U.prompt64(qs, k[:, :1], v[:, :1], [m], [m], True, d ** -0.5), "prompt")
    with pytest.raises(df11.DF11Error):
        wide = torch.as_strided(cache.k.view(-1), (m, 1, d), (2 ** 24, d, 1))
        df11.attend_prompt(qs, wide, wide, s, s, os)


# ------------------------------------------------------- streams, graphs, order

def _one_of_each(seed):
    """Inputs and a function that enqueues all four operators on a stream."""
    lens, ps, h, hk, d = [300, 1, 77], 16, 8, 2, 128
    q_lens = [20, 1, 77]
    n = sum(q_lens)
    t, n_pages = U.make_tables(lens, ps, seed)
    pages = t.to(DEV)
    cache = df11.kv_cache(n_pages, hk, ps, d, int8=True)
    cache.k.random_(-127, 128, generator=torch.Generator(DEV).manual_seed(seed))
    cache.v.copy_(cache.k.flip(0))
    for x in (cache.k_scale, cache.v_scale):
        x.fill_(0.02)
    q, k, v = _rand((n, h, d), seed), _rand((n, hk, d), seed + 1), _rand((n, hk, d), seed + 2)
    new = torch.cat([torch.arange(b - a, b) for a, b in zip(q_lens, lens)])
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(q_lens))
    slots = (t[seq, new // ps].long() * ps + new % ps).to(DEV)
    starts, q_starts = U.starts_of(lens).to(DEV), U.starts_of(q_lens).to(DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, out1 = torch.empty_like(q), torch.empty(3, h, d, dtype=torch.bfloat16, device=DEV)
    kd, vd = (torch.empty(sum(lens), hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def go(stream=None):
        df11.kv_write(cache, k, v, slots, stream=stream)
        df11.kv_read(cache, pages, starts, kd, vd, stream=stream)
        df11.attend_prompt(q, kd, vd, q_starts, starts, out, stream=stream)
        df11.attend_token(q[:3], cache, pages, ln, out1, stream=stream)

    return go, (kd, vd, out, out1), (q, k, v)


def test_streams_and_repeats():
    log("streams")
    go, outs, _ = _one_of_each(81)
    go()
    torch.cuda.synchronize()
    first = [x.clone() for x in outs]
    for stream in (torch.cuda.Stream(), torch.cuda.Stream()):
        for x in outs:
            x.fill_(3.0)
        torch.cuda.synchronize()
        go(stream)
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, first))


def test_graph_replays():
    log("graph")
    go, outs, (q, k, v) = _one_of_each(91)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for i in range(4):
        q.copy_(_rand(q.shape, 100 + i))
        k.copy_(_rand(k.shape, 200 + i))
        for x in outs:
            x.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        go()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, got)), i


# ------------------------------------------------------------------- refusals

def test_binding_refuses():
    log("refusals")
    hk, d, ps = 2, 64, 16
    cache, pages = _cache([40, 40], ps, hk, d, False, 61)
    q8, _ = _cache([40, 40], ps, hk, d, True, 61)
    q = _rand((2, 4, d), 1)
    out, ln = torch.empty_like(q), torch.tensor([40, 40], dtype=torch.int32, device=DEV)
    k, s = _rand((5, hk, d), 2), torch.arange(5, device=DEV)
    starts = U.starts_of([2, 3]).to(DEV)
    bad = [
        lambda: df11.attend_token(q.cpu(), cache, pages, ln, out),
        lambda: df11.attend_token(q.float(), cache, pages, ln, out),
        lambda: df11.attend_token(q[:, :, ::2], cache, pages, ln, out),
        lambda: df11.attend_token(q, cache, pages.long(), ln, out),
        lambda: df11.attend_token(q, cache, pages[:1], ln, out),
        lambda: df11.attend_token(q, cache, pages, ln.long(), out),
        lambda: df11.attend_token(q, cache, pages, ln[:1], out),
        lambda: df11.attend_token(q, cache, pages, ln, out[:1]),
        lambda: df11.attend_token(q, cache, pages, ln, out[:, :3]),
        lambda: df11.attend_token(q[:, :3], cache, pages, ln, out[:, :3]),                       # heads % kv_heads
        lambda: df11.attend_token(q, df11.KVCache(q8.k, q8.v), pages, ln, out),                  # no scales
        lambda: df11.attend_token(q, df11.KVCache(cache.k, cache.v, q8.k_scale, q8.v_scale), pages, ln, out),
        lambda: df11.attend_token(q, df11.KVCache(cache.k, cache.v[:1]), pages, ln, out),
        lambda: df11.attend_token(q, df11.KVCache(cache.k.float(), cache.v.float()), pages, ln, out),
        lambda: df11.attend_token(q, df11.KVCache(cache.k[:, :, :8].contiguous(), cache.v[:, :, :8].contiguous()), pages, ln, out),
        lambda: df11.attend_token(q, cache, pages, ln, out, scale=0.0),
        lambda: df11.attend_token(q, cache, pages, ln, out, scale=math.nan),
        lambda: df11.attend_token(q, cache, pages, ln, out, scale=-1.0),
        lambda: df11.attend_token(q, cache, pages, ln, q[:, :1].expand(2, 4, d)),                # overlapping output
        lambda: df11.kv_write(cache, k, k[:4], s),
        lambda: df11.kv_write(cache, k, k, s[:4]),
        lambda: df11.kv_write(cache, k, k, s.int()),
        lambda: df11.kv_write(cache, k[:, :1], k[:, :1], s),
        lambda: df11.kv_read(cache, pages, starts[:2], k, k.clone()),
        lambda: df11.kv_read(cache, pages, starts, k, k[:4]),
        lambda: df11.attend_prompt(k, k, k[:4], starts, starts, k.clone()),
        lambda: df11.attend_prompt(k, k, k, starts, starts[:2], k.clone()),
        lambda: df11.attend_prompt(k, k, k, starts.long(), starts, k.clone()),
        lambda: df11.attend_prompt(k[:, :1], k, k, starts, starts, k[:, :1].clone()),            # heads % kv_heads
        lambda: df11.attend_prompt(k.float(), k, k, starts, starts, k.clone()),
        lambda: df11.attend_prompt(k[:, :, :32], k[:, :, :32], k[:, :, :32], starts, starts, k[:, :, :32].clone()),
        lambda: df11.attend_prompt(k, k, k, starts, starts, k.clone(), scale=math.inf),
        lambda: df11.attend_prompt(k, k, k, starts, starts, k.cpu()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, df11.DF11Error)):
            f()
            raise AssertionError(f"call {i} was accepted")


def test_empty_calls():
    log("empty calls")
    cache = df11.kv_cache(2, 1, 16, 64)
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)   # noqa: E731
    df11.kv_write(cache, e, e, torch.empty(0, dtype=torch.int64, device=DEV))
    df11.kv_read(cache, torch.empty(0, 1, dtype=torch.int32, device=DEV), i32(0), e, e)
    df11.attend_prompt(e, e, e, i32(0), i32(0), e)
    df11.attend_token(e, cache, torch.empty(0, 1, dtype=torch.int32, device=DEV), i32(), e)
    out = torch.full((3, 1, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    df11.attend_prompt(_rand((3, 1, 64), 1), e, e, i32(0, 3), i32(0, 0), out)
    assert bool((out == 0).all())
