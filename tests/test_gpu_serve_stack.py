"""The decoder stack of serve.py end to end: compressed weights decoded by the
layer loop, keys and values written to the paged cache, prompts, a second piece
behind the first and single tokens, against a plain stack in 32 bits that keeps
every key and value and sees each sequence whole."""
import numpy as np
import pytest
import torch

from lossless_bf16_weight_amd import serve
from lossless_bf16_weight_amd import workloads as W

from gpu_util import log

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, D, FFN, LAYERS = 256, 6, 2, 64, 512, 2
SHAPES = [(HEADS * D, HIDDEN), (KV * D, HIDDEN), (KV * D, HIDDEN), (HIDDEN, HEADS * D), (FFN, HIDDEN), (FFN, HIDDEN),
          (HIDDEN, FFN)]


def _plain(x, layers):
    """One whole sequence [n, HIDDEN] through the stack in 32 bits (CPU)."""
    n = x.shape[0]
    pos = torch.arange(n)
    for wq, wk, wv, wo, gate, up, down in layers:
        h = serve.norm(x)
        q, k, v = ((h @ w.T).view(n, -1, D) for w in (wq, wk, wv))
        q, k = serve.rotary(q, pos), serve.rotary(k, pos)
        k, v = (t.repeat_interleave(HEADS // KV, 1) for t in (k, v))
        s = torch.einsum("nhd,mhd->hnm", q, k) * D ** -0.5
        s = s.masked_fill(pos[None, None, :] > pos[None, :, None], -torch.inf)
        x = x + torch.einsum("hnm,mhd->nhd", s.softmax(-1), v).reshape(n, -1) @ wo.T
        h = serve.norm(x)
        x = x + (torch.nn.functional.silu(h @ gate.T) * (h @ up.T)) @ down.T
    return x


@pytest.mark.parametrize("int8", [False, True])
def test_stack_against_a_plain_one(int8):
    log(f"decoder stack, int8 cache {int8}")
    words = [[W.normal_bf16(s, seed=10 * l + i, std=0.06) for i, s in enumerate(SHAPES)] for l in range(LAYERS)]
    layers = [[torch.from_numpy(w.astype(np.uint32).view(np.int32) << 16).view(torch.float32) for w in ws] for ws in words]
    pieces, steps = [[5, 70, 1], [33, 1, 40]], 4
    total = [a + b + steps for a, b in zip(*pieces)]
    gen = torch.Generator().manual_seed(3)
    xs = [torch.randn(n, HIDDEN, generator=gen).to(torch.bfloat16) for n in total]
    stack = serve.DecoderStack(serve.compressed_layers(words), HEADS, KV, D, 3, n_pages=24, page_size=16, max_len=128, int8=int8)
    got = [[] for _ in xs]
    at = [0, 0, 0]
    for new in pieces + [[1, 1, 1]] * steps:
        rows = torch.cat([x[a:a + n] for x, a, n in zip(xs, at, new)]).to("cuda")
        out = (stack.token(rows) if new == [1, 1, 1] else stack.prompt(rows, new)).float().cpu()
        for s, part in enumerate(out.split(new)):
            got[s].append(part)
        at = [a + n for a, n in zip(at, new)]
    assert stack.lens == total
    # About 14 roundings to BF16 a layer lie on the way to an output, each at
    # most 2^-8 of what it rounds and independent of the others; 8-bit keys
    # and values are off by at most 1/254 of their row's largest, about 4
    # times the row's root mean square: 2 x 4 / 254 more.
    bound = LAYERS * (14 * 2.0 ** -8 + (8 / 254 if int8 else 0))
    for x, parts in zip(xs, got):
        want = _plain(x.float(), layers)
        off = (torch.cat(parts) - want).norm(dim=-1) / want.norm(dim=-1)
        assert float(off.max()) < bound, (float(off.max()), bound)


def test_stack_refuses_what_does_not_fit():
    words = [[W.normal_bf16(s, seed=i, std=0.06) for i, s in enumerate(SHAPES)]]
    stack = serve.DecoderStack(serve.compressed_layers(words), HEADS, KV, D, 1, n_pages=2, page_size=16, max_len=64)
    x = torch.zeros(33, HIDDEN, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError):
        stack.prompt(x, [33])
