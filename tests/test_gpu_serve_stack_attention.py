"""Every attention call of a decoder stack (serve.py) against its definition in
64 bits, over all keys and values that the layer has made for the sequence so
far: positions, slots, pages and lengths of each pass, within the operators' own
bounds (the bound of the whole stack's result is wide)."""
import pytest
import torch

from lossless_bf16_weight_amd import serve
from lossless_bf16_weight_amd import workloads as W

import serve_precision as P
import serve_util as U
from gpu_util import log
from test_gpu_serve_stack import D, HEADS, HIDDEN, KV, SHAPES

pytestmark = pytest.mark.gpu


class _Watch:
    """Stands before the operators in serve.py: keeps what is written, and
    checks what attention gives."""

    def __init__(self, patch, n_seqs, int8):
        self.int8, self.made, self.new, self.calls = int8, {}, None, 0
        self.n_seqs = n_seqs
        self.last = None
        for name in ("kv_write", "attend_prompt", "attend_token"):
            self.patch(patch, name)

    def patch(self, patch, name):
        before, real = getattr(self, name), getattr(serve, name)

        def call(*args, **kw):
            got = real(*args, **kw)
            torch.cuda.synchronize()
            before(*args, **kw)
            return got
        patch.setattr(serve, name, call)

    def kv_write(self, cache, k, v, slots):
        rows = self.made.setdefault(cache.k.data_ptr(), [[] for _ in range(self.n_seqs)])
        for s, (a, b) in enumerate(zip(k.cpu().split(self.new), v.cpu().split(self.new))):
            rows[s].append((a, b))
        self.last = [tuple(torch.cat(x) for x in zip(*parts)) for parts in rows]

    def read(self, rows, rounded):
        """What the cache gives back of BF16 rows, in 64 bits."""
        if not self.int8:
            return rows.double()
        codes, scales = U.quantise32(rows)
        if rounded:
            return (codes.float() * scales[..., None]).to(torch.bfloat16).double()
        return codes.double() * scales.double()[..., None]

    def attend_prompt(self, q, k, v, q_starts, k_starts, out):
        lens = [len(a) for a, _ in self.last]
        cached = lens != self.new
        k64, v64 = (torch.cat([self.read(x[i], True) if cached else x[i].double() for x in self.last]) for i in (0, 1))
        U.within(out, *U.prompt64(q, k64, v64, self.new, lens, True, D ** -0.5), (self.new, lens))
        self.calls += 1

    def attend_token(self, q, cache, pages, lens, out):
        q = q.double().cpu()
        for s, rows in enumerate(self.last):
            k64, v64 = (self.read(x, False) for x in rows)
            for h in range(HEADS):
                g = h // (HEADS // KV)
                U.within(out[s, h], *P.attend64(q[s, h], k64[:, g], v64[:, g], D ** -0.5), (s, h))
        self.calls += 1


@pytest.mark.parametrize("int8", [False, True])
def test_attention_of_every_pass(int8, monkeypatch):
    log(f"decoder stack, attention of every pass, int8 cache {int8}")
    layers, n_seqs = 2, 3
    words = [[W.normal_bf16(s, seed=10 * l + i, std=0.06) for i, s in enumerate(SHAPES)] for l in range(layers)]
    stack = serve.DecoderStack(serve.compressed_layers(words), HEADS, KV, D, n_seqs, n_pages=24, page_size=16, max_len=128, int8=int8)
    watch = _Watch(monkeypatch, n_seqs, int8)
    gen = torch.Generator(device="cuda").manual_seed(13)
    passes = [[5, 70, 1], [0, 16, 31], [1, 1, 1], [33, 0, 2], [1, 1, 1], [1, 1, 1]]
    for new in passes:
        x = torch.randn(sum(new), HIDDEN, device="cuda", generator=gen).to(torch.bfloat16)
        watch.new = new
        stack.token(x) if new == [1, 1, 1] else stack.prompt(x, new)
    assert watch.calls == layers * len(passes)
