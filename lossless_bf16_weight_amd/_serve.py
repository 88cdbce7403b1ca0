"""Binding of the serving operators of libdf11.so (C ABI in include/df11.h):
a paged key-value cache, as BF16 words or in 8 bits, attention over packed
prompts, and attention of one new token of each sequence over the cache.

They are what a consumer of the layer loop (jit.LayerLoop) needs beside its
products with the decoded weights.  Argument marshalling only: what the C ABI
cannot see behind a device pointer (devices, dtypes, shapes) is checked here
and raises ValueError; the library checks the rest and raises DF11Error.
Calls enqueue on `stream` (the current one by default) and return.
"""
from __future__ import annotations

import math
import struct
from functools import lru_cache
from typing import NamedTuple, Optional

import torch

from ._lib import OK, _raise, lib

BF16, INT8, F32, I32, I64 = torch.bfloat16, torch.int8, torch.float32, torch.int32, torch.int64
KV_BF16, KV_INT8 = 0, 1
ROTATE_NEIGHBOURS = 1
ATTEND_CAUSAL = 1

# The argument structs of include/df11.h, field by field.
_CACHE = "QQQQIIIIII"
_TABLE = "QqII"
_ROWS = "Qqq"
_WRITE = struct.Struct("<" + _CACHE + 2 * _ROWS + "QQ")
_ROTATION = "QQQqIIIf"
_HEADS = struct.Struct("<" + _ROTATION + 4 * _ROWS + "QQQIIIf")
_APPEND = struct.Struct("<" + _CACHE + _ROTATION + 5 * _ROWS + "QQQQIf")
_READ = struct.Struct("<" + _CACHE + _TABLE + 2 * _ROWS + "QQII")
_TOKEN = struct.Struct("<" + _CACHE + _TABLE + 2 * _ROWS + "QQQIIfI")
_TOKEN_WINDOW = struct.Struct(_TOKEN.format + "II")
_PROMPT = struct.Struct("<" + 4 * _ROWS + "QQQQQQIIIIIf")

_CHUNK = struct.Struct("<" + _CACHE + _TABLE + 2 * _ROWS + "QQQQQIIIIIf")


class KVCache(NamedTuple):
    """A paged key-value cache: k and v are [n_pages, n_kv_heads, page_size,
    head_dim] tensors of bfloat16, or of int8 with float32 scales [n_pages,
    n_kv_heads, page_size] (an element is code * scale).  page_size is a power
    of two from 16 to 1024, head_dim 64 or 128.  Slot page * page_size + i is
    position i of a page."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None


def kv_cache(n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, int8: bool = False, device="cuda") -> KVCache:
    """A cache of zeros, of BF16 words or (int8) of 8-bit codes and scales."""
    shape = (n_pages, n_kv_heads, page_size, head_dim)
    dtype = torch.int8 if int8 else torch.bfloat16
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if not int8:
        return KVCache(k, v)
    return KVCache(k, v, *(torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))


def _cache_fields(c: KVCache):
    k, v, ks, vs = c
    if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor) or not k.is_cuda or k.dim() != 4:
        raise ValueError("cache: CUDA tensors [n_pages, n_kv_heads, page_size, head_dim] are needed")
    dev, shape, dtype = k.get_device(), k.shape, k.dtype
    if v.shape != shape or v.dtype is not dtype or v.get_device() != dev:
        raise ValueError("cache: k and v differ in shape, dtype or device")
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("cache: the pages must be contiguous")
    if dtype is BF16:
        if ks is not None or vs is not None:
            raise ValueError("cache: scales go with int8 pages")
        a, b, store = 0, 0, KV_BF16
    elif dtype is INT8:
        for s in (ks, vs):
            if s is None or s.shape != shape[:3] or s.dtype is not F32 or s.get_device() != dev or not s.is_contiguous():
                raise ValueError("cache: int8 pages need contiguous float32 scales [n_pages, n_kv_heads, page_size]")
        a, b, store = ks.data_ptr(), vs.data_ptr(), KV_INT8
    else:
        raise ValueError(f"cache: bfloat16 or int8 pages are needed, not {dtype}")
    n_pages, heads, page, d = shape
    return dev, heads, d, (k.data_ptr(), v.data_ptr(), a, b, n_pages, page, heads, d, store, 0)


def _rows(x: torch.Tensor, what: str, dev: int, d: int, n: int = -1, heads: int = -1):
    """(n, heads, fields) of a [rows, heads, head_dim] BF16 tensor."""
    if not isinstance(x, torch.Tensor) or x.dtype is not BF16 or x.dim() != 3 or x.get_device() != dev:
        raise ValueError(f"{what}: a bfloat16 tensor [rows, heads, head_dim] on cuda:{dev} is needed")
    rows, h, dim = x.shape
    s0, s1, s2 = x.stride()
    if dim != d or s2 != 1 or (n >= 0 and rows != n) or (heads >= 0 and h != heads):
        raise ValueError(f"{what}: shape {tuple(x.shape)}, strides {x.stride()}; "
                         f"[{n if n >= 0 else 'rows'}, {heads if heads >= 0 else 'heads'}, {d}] with a contiguous last dimension is needed")
    # (a stride that no element uses may be anything)
    return rows, h, (x.data_ptr(), s0 if rows > 1 else 0, s1 if h > 1 else 0)


def _index(x: torch.Tensor, what: str, dev: int, dtype, n: int):
    if not isinstance(x, torch.Tensor) or x.dtype is not dtype or x.dim() != 1 or x.get_device() != dev or x.shape[0] != n or not x.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} tensor [{n}] on cuda:{dev} is needed")
    return x.data_ptr()


def _table(pages: torch.Tensor, dev: int, n: int):
    if not isinstance(pages, torch.Tensor) or pages.dtype is not I32 or pages.dim() != 2 or pages.get_device() != dev or pages.shape[0] != n or (
            pages.shape[1] > 1 and pages.stride(1) != 1):
        raise ValueError(f"pages: an int32 tensor [{n}, entries] on cuda:{dev} with contiguous rows is needed")
    return pages.data_ptr(), pages.stride(0) if n > 1 else 0, pages.shape[1], 0


@lru_cache(maxsize=None)
def _device(dev: int) -> torch.device:
    return torch.device("cuda", dev)


def _workspace(need: int, given, dev: int, stream):
    """Pointer, bytes and the tensor that holds them (kept until the launch)."""
    if need == 0:
        return 0, 0, None
    if given is None:
        if stream is None:
            given = torch.empty(need, dtype=torch.uint8, device=_device(dev))
        else:
            with torch.cuda.stream(stream):    # (the allocator reuses it in this stream's order)
                given = torch.empty(need, dtype=torch.uint8, device=_device(dev))
    elif given.get_device() != dev or not given.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on cuda:{dev} is needed")
    return given.data_ptr(), given.numel() * given.element_size(), given


def _window(window: int, sinks: int):
    if window < 0 or sinks < 0:
        raise ValueError(f"window {window}, sinks {sinks}: numbers from 0 are needed")
    return min(window, 2 ** 31), min(sinks, 2 ** 31)


def _launch(fn, args: bytes, dev: int, stream):
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)   # (torch.cuda.current_stream(dev).cuda_stream, 1 us sooner)
    else:
        handle = stream.cuda_stream
    st = fn(args, dev, handle)
    if st != OK:
        _raise(st)


def kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None):
    """Write token t's keys and values (rows t of k and v, [tokens, n_kv_heads,
    head_dim] bfloat16) into slot slots[t] (int64) of the cache, quantised on
    the way where its pages are int8.  A slot outside the cache, such as -1,
    leaves its token out; the others are distinct."""
    dev, heads, d, c = _cache_fields(cache)
    n, _, kr = _rows(k, "k", dev, d, heads=heads)
    _, _, vr = _rows(v, "v", dev, d, n, heads)
    _launch(lib().df11_kv_write, _WRITE.pack(*c, *kr, *vr, _index(slots, "slots", dev, I64, n), n), dev, stream)


class Rotation:
    """The position rotation of a head's first 2 * len(turns) elements (made by
    rotation()).  turns: int64 [pairs], frequencies as fractions of a turn a
    position, times 2^64; axes: uint8 [pairs], the axis of each pair, or None;
    n_axes: how many a position has.  What it holds is checked here, once, and
    does not change."""
    __slots__ = ("turns", "axes", "n_axes", "interleaved", "factor", "_device", "_fields")

    def __init__(self, turns: torch.Tensor, axes: Optional[torch.Tensor] = None, n_axes: int = 1, interleaved: bool = False, factor: float = 1.0):
        if turns.dtype is not I64 or turns.dim() != 1 or not turns.is_contiguous():
            raise ValueError("rotation: contiguous int64 turns [pairs] are needed")
        if axes is not None and (axes.dtype is not torch.uint8 or axes.shape != turns.shape or axes.device != turns.device or not axes.is_contiguous()):
            raise ValueError("rotation: axes must be contiguous uint8 [pairs] on the turns' device")
        fields = (turns.data_ptr(), 0 if axes is None else axes.data_ptr()), (turns.shape[0], ROTATE_NEIGHBOURS if interleaved else 0, float(factor))
        for name, value in zip(self.__slots__, (turns, axes, int(n_axes), bool(interleaved), float(factor), turns.get_device(), fields)):
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError("a Rotation does not change")


def rotation(rotary_dim: int, base: float = 10000.0, freqs=None, axes=None, interleaved: bool = False, factor: float = 1.0,
             device="cuda") -> Rotation:
    """A rotation of the first rotary_dim elements of a head (a multiple of 16,
    0 for none): pair i turns by position * freqs[i] radians, freqs[i] being
    base ** (-2 i / rotary_dim) unless given.  Pairs are elements i and i +
    rotary_dim / 2, or (interleaved) neighbours.  axes: for positions with
    several axes (time, height, width ...; up to 4), the axis of each pair.
    factor multiplies the rotated elements."""
    pairs = rotary_dim // 2
    if rotary_dim % 16 or rotary_dim < 0:
        raise ValueError(f"rotary_dim {rotary_dim}: a multiple of 16 is needed")
    f = [base ** (-i / pairs) for i in range(pairs)] if freqs is None else [float(x) for x in freqs]
    if len(f) != pairs or not all(map(math.isfinite, f)) or not math.isfinite(factor):
        raise ValueError(f"freqs, factor: {pairs} finite frequencies and a finite factor are needed")
    turns = [round(math.fmod(x / (2 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64 for x in f]
    n_axes = 1
    if axes is not None:
        axes = [int(x) for x in axes]
        if len(axes) != pairs or not all(0 <= x < 4 for x in axes):
            raise ValueError(f"axes: {pairs} numbers from 0 to 3 are needed")
        n_axes = max(axes, default=0) + 1
    return Rotation(torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in turns], dtype=I64, device=device),
                    torch.tensor(axes, dtype=torch.uint8, device=device) if n_axes > 1 else None, n_axes, bool(interleaved), float(factor))


def _rotation_fields(r: Optional[Rotation], positions, dev: int, n: int):
    if r is None or r._fields[1][0] == 0:
        return 0, 0, 0, 0, 0, 0, 0, 0.0
    (turns, axes), (pairs, flags, factor) = r._fields
    p, n_axes = positions, r.n_axes
    if r._device != dev:
        raise ValueError(f"rotation: on cuda:{r._device}, not cuda:{dev}")
    if not isinstance(p, torch.Tensor) or p.dtype is not I32 or p.get_device() != dev or p.dim() not in (1, 2) or p.shape[0] != n:
        raise ValueError(f"positions: an int32 tensor [{n}] or [{n}, axes] on cuda:{dev} is needed")
    if p.dim() == 2:
        if not n_axes <= p.shape[1] <= 4 or (p.shape[1] > 1 and p.stride(1) != 1):
            raise ValueError(f"positions: shape {tuple(p.shape)}, strides {p.stride()}; {n_axes} to 4 axes, contiguous in a row, are needed")
        n_axes = p.shape[1]
    elif n_axes > 1:
        raise ValueError(f"positions: [{n}, {n_axes}] is needed")
    return turns, axes, p.data_ptr(), p.stride(0) if n > 1 else 0, pairs, n_axes, flags, factor


def _weight(w, what: str, dev: int, d: int):
    if w is None:
        return 0
    if not isinstance(w, torch.Tensor) or w.dtype is not BF16 or w.shape != (d,) or w.get_device() != dev or not w.is_contiguous():
        raise ValueError(f"{what}: a contiguous bfloat16 tensor [{d}] on cuda:{dev} is needed")
    return w.data_ptr()


_NO_ROWS = 0, 0, (0, 0, 0)


def rotate_heads(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: Optional[torch.Tensor], rotation: Optional[Rotation],
                 q_out: Optional[torch.Tensor], k_out: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None):
    """Queries and keys ([tokens, heads, head_dim] bfloat16; either may be None)
    with each head normed, x * weight / sqrt(mean(x^2) + eps), where its weight
    ([head_dim] bfloat16) is given, and rotated by the token's position, into
    q_out and k_out (which may be q and k).  positions: int32 [tokens], or
    [tokens, axes].  rotation None: the norms alone."""
    x = k if q is None else q
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 3:
        raise ValueError("q, k: CUDA tensors [tokens, heads, head_dim] are needed")
    dev, (n, _, d) = x.get_device(), x.shape
    _, h, qr = _NO_ROWS if q is None else _rows(q, "q", dev, d, n)
    _, hk, kr = _NO_ROWS if k is None else _rows(k, "k", dev, d, n)
    _, _, qo = _NO_ROWS if q is None else _rows(q_out, "q_out", dev, d, n, h)
    _, _, ko = _NO_ROWS if k is None else _rows(k_out, "k_out", dev, d, n, hk)
    _launch(lib().df11_rotate_heads, _HEADS.pack(*_rotation_fields(rotation, positions, dev, n), *qr, *kr, *qo, *ko,
                                                 _weight(q_weight, "q_weight", dev, d), _weight(k_weight, "k_weight", dev, d), n, h, hk, d, eps),
            dev, stream)


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, positions: Optional[torch.Tensor], slots: torch.Tensor,
              rotation: Optional[Rotation], k_weight: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
              q_out: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
              eps: float = 1e-6, stream=None):
    """rotate_heads and kv_write in one launch: token t's keys normed and
    rotated into slot slots[t] (int64) of the cache, with its values as they
    are; queries, where given, into q_out; keys also as rows of k_out, where
    that is given.  Keys in 8 bits are quantised without rounding them to
    bfloat16 first.  A slot outside the cache leaves its token out of it."""
    dev, heads, d, c = _cache_fields(cache)
    n, _, kr = _rows(k, "k", dev, d, heads=heads)
    _, _, vr = _rows(v, "v", dev, d, n, heads)
    _, h, qr = _NO_ROWS if q is None else _rows(q, "q", dev, d, n)
    _, _, qo = _NO_ROWS if q is None else _rows(q_out, "q_out", dev, d, n, h)
    _, _, ko = _NO_ROWS if k_out is None else _rows(k_out, "k_out", dev, d, n, heads)
    _launch(lib().df11_kv_append, _APPEND.pack(*c, *_rotation_fields(rotation, positions, dev, n), *qr, *kr, *vr, *qo, *ko,
                                               _index(slots, "slots", dev, I64, n), _weight(q_weight, "q_weight", dev, d),
                                               _weight(k_weight, "k_weight", dev, d), n, h, eps), dev, stream)


def kv_read(cache: KVCache, pages: torch.Tensor, starts: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor, stream=None):
    """Read back the first starts[s + 1] - starts[s] tokens of each sequence as
    packed bfloat16 rows starts[s] .. of k_out and v_out ([tokens, n_kv_heads,
    head_dim]).  pages: int32 [sequences, entries], starts: int32 [sequences +
    1]."""
    dev, heads, d, c = _cache_fields(cache)
    n, _, kr = _rows(k_out, "k_out", dev, d, heads=heads)
    _, _, vr = _rows(v_out, "v_out", dev, d, n, heads)
    seqs = pages.shape[0]
    _launch(lib().df11_kv_read, _READ.pack(*c, *_table(pages, dev, seqs), *kr, *vr,
                                           _index(starts, "starts", dev, I32, seqs + 1), n, seqs, 0), dev, stream)


@lru_cache(maxsize=4096)
def token_workspace(n_seqs: int, n_heads: int, n_kv_heads: int, head_dim: int, page_size: int, entries: int, device: int = 0,
                    window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace that attend_token needs for these sizes (`entries`:
    the page table's width)."""
    args = _TOKEN_WINDOW.pack(0, 0, 0, 0, 1, page_size, n_kv_heads, head_dim, 0, 0, 0, 0, entries, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0,
                              n_seqs, n_heads, 1.0, 0, *_window(window, sinks))
    return lib().df11_attend_token_window_workspace(args, device)


def attend_token(q: torch.Tensor, cache: KVCache, pages: torch.Tensor, lens: torch.Tensor, out: torch.Tensor, scale=None,
                 workspace: Optional[torch.Tensor] = None, stream=None, window: int = 0, sinks: int = 0):
    """Attention of one query row a sequence (q, out: [sequences, n_heads,
    head_dim] bfloat16) over the first lens[s] (int32) positions of its pages
    (int32 [sequences, entries]); with a window above 0 over the last `window`
    of them and the first `sinks`.  scale: 1 / sqrt(head_dim) by default.
    workspace: at least token_workspace() bytes that no other call uses
    meanwhile; by default taken from torch's allocator."""
    dev, hk, d, c = _cache_fields(cache)
    n, h, qr = _rows(q, "q", dev, d)
    _, _, orow = _rows(out, "out", dev, d, n, h)
    t = _table(pages, dev, n)
    at = _index(lens, "lens", dev, I32, n)
    if scale is None:
        scale = d ** -0.5
    if window or sinks:
        window, sinks = _window(window, sinks)
        p, size, keep = _workspace(token_workspace(n, h, hk, d, c[5], t[2], dev, window, sinks), workspace, dev, stream)
        _launch(lib().df11_attend_token_window, _TOKEN_WINDOW.pack(*c, *t, *qr, *orow, at, p, size, n, h, scale, 0, window, sinks), dev, stream)
        return
    p, size, keep = _workspace(token_workspace(n, h, hk, d, c[5], t[2], dev), workspace, dev, stream)
    _launch(lib().df11_attend_token, _TOKEN.pack(*c, *t, *qr, *orow, at, p, size, n, h, scale, 0), dev, stream)


@lru_cache(maxsize=4096)
def prompt_workspace(n_q: int, n_k: int, n_seqs: int, n_heads: int, n_kv_heads: int, head_dim: int, device: int = 0) -> int:
    """Bytes of workspace that attend_prompt needs for these sizes."""
    args = _PROMPT.pack(*(12 * (0,)), 0, 0, 0, 0, n_q, n_k, n_seqs, n_heads, n_kv_heads, head_dim, 0, 1.0)
    return lib().df11_attend_prompt_workspace(args, device)


def attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_starts: torch.Tensor, k_starts: torch.Tensor,
                  out: torch.Tensor, causal: bool = True, scale=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of packed sequences: queries q_starts[s] .. q_starts[s + 1] - 1
    (rows of q, [rows, n_heads, head_dim] bfloat16) over keys and values
    k_starts[s] .. (rows of k and v, [rows, n_kv_heads, head_dim]) into the same
    rows of out.  causal: the queries are the last of their sequence, query i
    sees the keys j <= i + n_keys - n_queries.  A row that sees no key is zero.
    starts: int32 [sequences + 1].  scale, workspace: as for attend_token."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
        raise ValueError("q: a CUDA tensor [rows, heads, head_dim] is needed")
    dev, d = q.get_device(), q.shape[2]
    n, h, qr = _rows(q, "q", dev, d)
    m, hk, kr = _rows(k, "k", dev, d)
    _, _, vr = _rows(v, "v", dev, d, m, hk)
    _, _, orow = _rows(out, "out", dev, d, n, h)
    seqs = q_starts.shape[0] - 1
    if seqs < 0:
        raise ValueError("q_starts: one entry more than sequences is needed")
    a, b = _index(q_starts, "q_starts", dev, I32, seqs + 1), _index(k_starts, "k_starts", dev, I32, seqs + 1)
    p, size, keep = _workspace(prompt_workspace(n, m, seqs, h, hk, d, dev), workspace, dev, stream)
    _launch(lib().df11_attend_prompt, _PROMPT.pack(*qr, *kr, *vr, *orow, a, b, p, size, n, m, seqs, h, hk, d,
                                                   ATTEND_CAUSAL if causal else 0, d ** -0.5 if scale is None else scale), dev, stream)


@lru_cache(maxsize=4096)
def chunk_workspace(n_q: int, n_seqs: int, n_heads: int, n_kv_heads: int, head_dim: int, page_size: int, entries: int, window: int = 0,
                    sinks: int = 0, device: int = 0) -> int:
    """Bytes of workspace that attend_chunk needs for these sizes (`entries`:
    the page table's width)."""
    args = _CHUNK.pack(0, 0, 0, 0, 1, page_size, n_kv_heads, head_dim, 0, 0, 0, 0, entries, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, n_q,
                       n_seqs, n_heads, ATTEND_CAUSAL, window, sinks, 1.0)
    return lib().df11_attend_chunk_workspace(args, device)


def attend_chunk(q: torch.Tensor, cache: KVCache, pages: torch.Tensor, q_starts: torch.Tensor, lens: torch.Tensor, out: torch.Tensor,
                 causal: bool = True, window: int = 0, sinks: int = 0, scale=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of a chunk of new tokens of each sequence: queries q_starts[s]
    .. q_starts[s + 1] - 1 (rows of q, [rows, n_heads, head_dim] bfloat16) over
    the first lens[s] (int32) positions of its pages (int32 [sequences,
    entries]), the new tokens' among them, into the same rows of out.  causal:
    query i of n stands at position p = lens[s] - n + i and sees the keys j <=
    p, with a window above 0 of these only j > p - window and the first `sinks`.
    A row that sees no key is zero; rows behind the last sequence are left
    alone.  starts: int32 [sequences + 1].  scale, workspace: as for
    attend_token.  The table's width is taken for how long a single sequence
    is: give the columns in use, pages[:, :entries]."""
    dev, hk, d, c = _cache_fields(cache)
    n, h, qr = _rows(q, "q", dev, d)
    _, _, orow = _rows(out, "out", dev, d, n, h)
    seqs = lens.shape[0]
    t = _table(pages, dev, seqs)
    a, b = _index(q_starts, "q_starts", dev, I32, seqs + 1), _index(lens, "lens", dev, I32, seqs)
    window, sinks = _window(window, sinks)
    p, size, keep = _workspace(chunk_workspace(n, seqs, h, hk, d, c[5], t[2], window, sinks, dev), workspace, dev, stream)
    _launch(lib().df11_attend_chunk, _CHUNK.pack(*c, *t, *qr, *orow, a, b, p, size, n, seqs, h, ATTEND_CAUSAL if causal else 0, window, sinks,
                                                 d ** -0.5 if scale is None else scale), dev, stream)
