"""rotate_heads and kv_append on the GPU against their definition in 64 bits,
within the bounds of serve_heads_util.py, and against kv_write bit for bit."""
import itertools

import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_heads_util as HU
import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
FILL = 7.0


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def _positions(n, axes, seed, far=False):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, 5000, (n, axes), generator=g, dtype=torch.int64)
    odd = [0, 1, 2 ** 31 - 1, -2 ** 31, -1, 131071, 2 ** 28 + 1] if far else [0]
    for i, x in enumerate(odd[:n]):
        p[i % n, i % axes] = x
    return p.to(torch.int32)


class _Case:
    def __init__(self, n, h, hk, d, rotary_dim, neighbours, axes, norms, seed=0, factor=1.0, far=False, base=10000.0):
        self.n, self.h, self.hk, self.d, self.neighbours, self.factor = n, h, hk, d, neighbours, factor
        fused = _rand((n, h + 2 * hk, d), seed).to(DEV)
        self.q, self.k, self.v = fused[:, :h], fused[:, h:h + hk], fused[:, h + hk:]
        self.positions = _positions(n, axes, seed + 1, far)
        pairs = rotary_dim // 2
        self.axes = [(3 * i) % axes for i in range(pairs)]
        self.freqs = HU.freqs64(rotary_dim, base)
        self.rotation = df11.rotation(rotary_dim, base=base, axes=self.axes if axes > 1 else None, interleaved=neighbours, factor=factor)
        self.p = (self.positions[:, 0].contiguous() if axes == 1 else self.positions).to(DEV)
        self.wq, self.wk = ((1 + 0.3 * _rand((d,), seed + 2 + i).float()).to(torch.bfloat16).to(DEV) if norms else None for i in range(2))

    def want(self, x, w, eps=1e-6):
        return HU.heads64(x, self.positions, self.freqs, self.axes, self.neighbours, self.factor, w, eps)

    def check(self, got, x, w, what):
        y, err = self.want(x, w)
        U.within(got, y, HU.bound_of(y, err), what)


def _guarded(n, heads, d):
    """Rows with unused rows, heads and words around them, and a check that those keep what they held."""
    whole = torch.full((n + 4, heads + 2, d + 8), FILL, dtype=torch.bfloat16, device=DEV)
    inside = whole[2:n + 2, 1:heads + 1, :d]

    def untouched():
        kept = whole.clone()
        kept[2:n + 2, 1:heads + 1, :d] = FILL
        return bool((kept == FILL).all())
    return inside, untouched


SHAPES = [(1, 4, 2, 128), (3, 1, 1, 64), (7, 20, 1, 128), (33, 6, 2, 64), (130, 24, 24, 128), (17, 12, 4, 64)]
FORMS = list(itertools.product(("all", "half", 16), (False, True), (1, 3), (False, True)))


@pytest.mark.parametrize("part,neighbours,axes,norms", FORMS)
def test_rotate_heads(part, neighbours, axes, norms):
    for i, (n, h, hk, d) in enumerate(SHAPES):
        log(f"rotate_heads {part} neighbours {neighbours} axes {axes} norms {norms}: {n} tokens {h}/{hk} heads of {d}")
        r = {"all": d, "half": d // 2}.get(part, part)
        c = _Case(n, h, hk, d, r, neighbours, axes, norms, seed=10 * i, far=True)
        (qo, q_kept), (ko, k_kept) = _guarded(n, h, d), _guarded(n, hk, d)
        df11.rotate_heads(c.q, c.k, c.p, c.rotation, qo, ko, c.wq, c.wk)
        torch.cuda.synchronize()
        c.check(qo, c.q, c.wq, ("q", n, h, hk, d))
        c.check(ko, c.k, c.wk, ("k", n, h, hk, d))
        assert q_kept() and k_kept()


@pytest.mark.parametrize("n,h,hk,d", [(2000, 16, 2, 128), (9001, 3, 1, 64), (1, 300, 7, 64), (400, 70, 35, 128)])
def test_many_tokens_and_many_heads(n, h, hk, d):
    """Waves that take all rows of a token, a part of them, and several batches of them."""
    log(f"rotate_heads {n} tokens of {h}/{hk} heads of {d}")
    c = _Case(n, h, hk, d, d, False, 1, True, seed=3)
    qo, ko = torch.empty_like(c.q), torch.empty_like(c.k)
    df11.rotate_heads(c.q, c.k, c.p, c.rotation, qo, ko, c.wq, c.wk)
    torch.cuda.synchronize()
    c.check(qo, c.q, c.wq, "q")
    c.check(ko, c.k, c.wk, "k")


def test_one_of_queries_and_keys_in_place_and_a_factor():
    c = _Case(37, 5, 3, 128, 96, False, 2, True, seed=5, factor=1.37)
    q, k = c.q.clone(), c.k.clone()
    df11.rotate_heads(c.q, None, c.p, c.rotation, c.q, None, c.wq)         # (within the fused rows)
    df11.rotate_heads(None, c.k, c.p, c.rotation, None, c.k)               # (no norm)
    torch.cuda.synchronize()
    c.check(c.q, q, c.wq, "q")
    c.check(c.k, k, None, "k")


def test_norms_alone_and_neither():
    c = _Case(9, 4, 2, 64, 0, False, 1, True, seed=6)
    for rotation in (c.rotation, None):
        qo, ko = torch.empty_like(c.q), torch.empty_like(c.k)
        df11.rotate_heads(c.q, c.k, None, rotation, qo, ko, c.wq, None)
        torch.cuda.synchronize()
        c.check(qo, c.q, c.wq, "q")
        assert torch.equal(HU.bits(ko), HU.bits(c.k))


def test_position_zero_leaves_the_words():
    for d, neighbours in itertools.product((64, 128), (False, True)):
        c = _Case(5, 3, 2, d, d, neighbours, 1, False, seed=7)
        qo, ko = torch.empty_like(c.q), torch.empty_like(c.k)
        df11.rotate_heads(c.q, c.k, torch.zeros_like(c.p), c.rotation, qo, ko)
        torch.cuda.synchronize()
        assert torch.equal(qo, c.q) and torch.equal(ko, c.k)


def test_given_frequencies_and_far_positions_of_several_turns():
    """Frequencies above a turn a position and below zero, far positions: the
    phase is exact."""
    d, n = 64, 8
    freqs = [(-1.0) ** i * 40.0 * 0.9 ** i for i in range(d // 2)]
    c = _Case(n, 2, 1, d, d, True, 1, False, seed=8, far=True)
    c.freqs, c.rotation = freqs, df11.rotation(d, freqs=freqs, interleaved=True)
    qo, ko = torch.empty_like(c.q), torch.empty_like(c.k)
    df11.rotate_heads(c.q, c.k, c.p, c.rotation, qo, ko)
    torch.cuda.synchronize()
    c.check(qo, c.q, None, "q")
    c.check(ko, c.k, None, "k")


@pytest.mark.parametrize("scale", [2.0 ** 120, 2.0 ** 64, 2.0 ** -60, 2.0 ** -120, 0.0])
def test_norms_of_any_size(scale):
    """Squares that pass 32 bits on either side."""
    log(f"norms of values of {scale}")
    for d in (64, 128):
        c = _Case(6, 3, 2, d, d, False, 1, True, seed=9)
        q = (c.q.float() * scale).to(torch.bfloat16)
        q[2] = c.q[2]           # a row of ordinary size among them
        out = torch.empty_like(q)
        df11.rotate_heads(q, None, c.p, c.rotation, out, None, c.wq)
        torch.cuda.synchronize()
        c.check(out, q, c.wq, (d, scale))


def test_odd_values_stay_in_their_head():
    c = _Case(6, 4, 2, 128, 64, False, 1, True, seed=11)
    clean, odd = torch.empty_like(c.q), torch.empty_like(c.q)
    df11.rotate_heads(c.q, None, c.p, c.rotation, clean, None, c.wq)
    c.q[1, 2, 5], c.q[4, 0, 100], c.q[5, 3, 0] = float("nan"), float("inf"), -float("inf")
    df11.rotate_heads(c.q, None, c.p, c.rotation, odd, None, c.wq)
    torch.cuda.synchronize()
    hit = torch.zeros(6, 4, dtype=torch.bool, device=DEV)
    hit[1, 2] = hit[4, 0] = hit[5, 3] = True
    assert torch.equal(HU.bits(clean)[~hit], HU.bits(odd)[~hit])
    assert bool(torch.isnan(odd[1, 2]).all())
    y, err = c.want(c.q, c.wq)
    assert torch.equal(torch.isnan(y), torch.isnan(odd.double().cpu()))
    # without a norm only the pair is hit
    df11.rotate_heads(c.q, None, c.p, c.rotation, odd, None)
    torch.cuda.synchronize()
    assert int((~torch.isfinite(odd[5, 3])).sum()) == 2 and int((~torch.isfinite(odd[4, 0])).sum()) == 1


# ---------------------------------------------------------------- into the cache

def _slots(n, n_slots, seed, left_out=()):
    s = torch.randperm(n_slots, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int64)
    for i, x in left_out:
        if i < n:
            s[i] = x
    return s.to(DEV)


def _filled_cache(pages, hk, ps, d, int8):
    c = df11.kv_cache(pages, hk, ps, d, int8=int8)
    for x in c:
        if x is not None:
            x.fill_(3)
    return c


def _same_cache(a, b):
    return all(x is y is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("part,neighbours,axes,norms", [("all", False, 1, False), ("half", True, 3, True), (16, False, 2, True), ("all", True, 1, True)])
def test_kv_append(part, neighbours, axes, norms, int8):
    for i, (n, h, hk, d) in enumerate(SHAPES):
        log(f"kv_append {part} neighbours {neighbours} axes {axes} norms {norms} int8 {int8}: {n} tokens {h}/{hk} heads of {d}")
        r = {"all": d, "half": d // 2}.get(part, part)
        c = _Case(n, h, hk, d, r, neighbours, axes, norms, seed=100 + 10 * i)
        ps = 16 if i % 2 else 64
        pages = -(-n // ps) + 2
        slots = _slots(n, pages * ps, i, [(1, -1), (4, pages * ps), (5, 2 ** 40)])
        cache, plain = _filled_cache(pages, hk, ps, d, int8), _filled_cache(pages, hk, ps, d, int8)
        (qo, q_kept), (ko, k_kept) = _guarded(n, h, d), _guarded(n, hk, d)
        df11.kv_append(cache, c.k, c.v, c.p, slots, c.rotation, k_weight=c.wk, q=c.q, q_out=qo, q_weight=c.wq, k_out=ko)
        q2, k2 = torch.empty_like(c.q), torch.empty_like(c.k)
        df11.rotate_heads(c.q, c.k, c.p, c.rotation, q2, k2, c.wq, c.wk)
        df11.kv_write(plain, k2, c.v, slots)
        torch.cuda.synchronize()
        assert q_kept() and k_kept()
        assert torch.equal(HU.bits(qo), HU.bits(q2)) and torch.equal(HU.bits(ko), HU.bits(k2))
        c.check(qo, c.q, c.wq, "q")
        if not int8:
            assert _same_cache(cache, plain)
            continue
        assert torch.equal(cache.v, plain.v) and torch.equal(cache.v_scale, plain.v_scale)
        # keys: half a step from the 32-bit value, where the other form rounds it to BF16 first
        y, err = c.want(c.k, c.wk)
        at = slots.cpu()
        used = (at >= 0) & (at < pages * ps)
        at, y, err = at[used], y[used], err[used]
        codes, scales = cache.k.cpu()[at // ps, :, at % ps].double(), cache.k_scale.cpu()[at // ps, :, at % ps].double()
        top = y.abs().amax(-1).clamp_min(U.TINY)
        assert bool(((scales * 127 - top).abs() <= err.amax(-1) + 4 * U.E * top).all())
        assert bool(((codes * scales[..., None] - y).abs() <= scales[..., None] * (0.5 + 2.0 ** -14) + err).all())
        free = torch.ones(pages * ps, dtype=torch.bool)
        free[at] = False
        f = torch.arange(pages * ps)[free]
        assert bool((cache.k.cpu()[f // ps, :, f % ps] == 3).all() and (cache.k_scale.cpu()[f // ps, :, f % ps] == 3).all())


@pytest.mark.parametrize("int8", [False, True])
def test_append_without_rotation_is_kv_write(int8):
    for d in (64, 128):
        c = _Case(40, 2, 3, d, 0, False, 1, False, seed=60)
        c.k[3, 1, 4], c.k[7, 0, 1], c.v[9, 2, 0], c.v[2, 0, 3] = float("inf"), float("nan"), float("nan"), -float("inf")
        c.k[11] = 0
        c.k[12] *= 2.0 ** -120
        slots = _slots(40, 96, 1)
        a, b = _filled_cache(6, 3, 16, d, int8), _filled_cache(6, 3, 16, d, int8)
        df11.kv_append(a, c.k, c.v, None, slots, None)
        df11.kv_write(b, c.k, c.v, slots)
        torch.cuda.synchronize()
        assert _same_cache(a, b)


def test_append_keys_in_place():
    c = _Case(21, 4, 2, 128, 128, False, 1, False, seed=70)
    q, k = c.q.clone(), c.k.clone()
    cache, slots = _filled_cache(3, 2, 16, 128, False), _slots(21, 48, 2)
    df11.kv_append(cache, c.k, c.v, c.p, slots, c.rotation, q=c.q, q_out=c.q, k_out=c.k)
    torch.cuda.synchronize()
    c.check(c.q, q, None, "q")
    c.check(c.k, k, None, "k")
    assert torch.equal(cache.k[slots // 16, :, slots % 16], c.k) and torch.equal(cache.v[slots // 16, :, slots % 16], c.v)


@pytest.mark.parametrize("int8", [False, True])
def test_slots_past_32_bits(int8):
    """A cache of 2^25 rows a head of 128: byte offsets past 2^32."""
    log(f"append past 2^32 bytes, int8 {int8}")
    pages, hk, d, ps = (1 << 14) + 3, 2 if not int8 else 3, 128, 1024
    cache = df11.kv_cache(pages, hk, ps, d, int8=int8)
    assert cache.k.numel() * cache.k.element_size() > 1 << 32
    c = _Case(5, 2, hk, d, d, False, 1, False, seed=80)
    slots = torch.tensor([pages * ps - 1, 0, 5, pages * ps - 1024, 7 * ps], device=DEV)
    ko = torch.empty_like(c.k)
    df11.kv_append(cache, c.k, c.v, c.p, slots, c.rotation, k_out=ko)
    torch.cuda.synchronize()
    k, v = cache.k[slots // ps, :, slots % ps].float(), cache.v[slots // ps, :, slots % ps].float()
    if int8:
        k, v = k * cache.k_scale[slots // ps, :, slots % ps][..., None], v * cache.v_scale[slots // ps, :, slots % ps][..., None]
    # (8 bits: within a step of 1/127 of the largest)
    for got, want in ((k, ko), (v, c.v)):
        want = want.float()
        assert bool(((got - want).abs() <= (want.abs().amax(-1, keepdim=True) / 127 if int8 else 0)).all())


def test_no_tokens():
    c = _Case(4, 2, 1, 64, 64, False, 1, False, seed=90)
    cache = _filled_cache(1, 1, 16, 64, False)
    none = c.q[:0]
    df11.rotate_heads(none, c.k[:0], c.p[:0], c.rotation, none, c.k[:0])
    df11.kv_append(cache, c.k[:0], c.v[:0], c.p[:0], torch.empty(0, dtype=torch.int64, device=DEV), c.rotation)
    torch.cuda.synchronize()
    assert bool((cache.k == 3).all())
