"""A decoder stack with a rotation (serve.py): heads normed, rotated and
appended in one launch, prompts and pieces over the pages, windows with sinks,
against a plain stack in 32 bits that sees each sequence whole."""
import numpy as np
import pytest
import torch

import lossless_bf16_weight_amd as df11
from lossless_bf16_weight_amd import serve
from lossless_bf16_weight_amd import workloads as W

import serve_chunk_util as CU
import serve_heads_util as HU
from gpu_util import log
from test_gpu_serve_stack import D, HEADS, HIDDEN, KV, LAYERS, SHAPES

pytestmark = pytest.mark.gpu


def _plain(x, layers, norms, window, sinks):
    """One whole sequence [n, HIDDEN] through the stack in 32 bits (CPU)."""
    n = x.shape[0]
    pos = torch.arange(n)[:, None]
    seen = CU.seen64(n, n, True, window, sinks)
    for l, (wq, wk, wv, wo, gate, up, down) in enumerate(layers):
        h = serve.norm(x)
        q, k, v = ((h @ w.T).view(n, -1, D) for w in (wq, wk, wv))
        qw, kw = norms[l] if norms else (None, None)
        q, k = (HU.heads64(t, pos, HU.freqs64(D, 500000.0), [0] * (D // 2), False, weight=w)[0].float() for t, w in ((q, qw), (k, kw)))
        k, v = (t.repeat_interleave(HEADS // KV, 1) for t in (k, v))
        s = torch.einsum("nhd,mhd->hnm", q, k) * D ** -0.5
        s = s.masked_fill(~seen, -torch.inf)
        x = x + torch.einsum("hnm,mhd->nhd", s.softmax(-1), v).reshape(n, -1) @ wo.T
        h = serve.norm(x)
        x = x + (torch.nn.functional.silu(h @ gate.T) * (h @ up.T)) @ down.T
    return x


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("norms,window,sinks", [(False, 0, 0), (True, 0, 0), (True, 20, 3), (False, 33, 0)])
def test_stack_over_pages(norms, window, sinks, int8):
    log(f"decoder stack over pages, norms {norms}, window {window} sinks {sinks}, int8 cache {int8}")
    words = [[W.normal_bf16(s, seed=10 * l + i, std=0.06) for i, s in enumerate(SHAPES)] for l in range(LAYERS)]
    layers = [[torch.from_numpy(w.astype(np.uint32).view(np.int32) << 16).view(torch.float32) for w in ws] for ws in words]
    gen = torch.Generator().manual_seed(3)
    weights = [tuple((1 + 0.2 * torch.randn(D, generator=gen)).to(torch.bfloat16) for _ in range(2)) for _ in range(LAYERS)] if norms else None
    passes = [[5, 70, 1], [33, 1, 40], [1, 1, 1], [1, 1, 1], [1, 0, 17], [1, 1, 1]]
    total = [sum(p) for p in zip(*passes)]
    xs = [torch.randn(n, HIDDEN, generator=gen).to(torch.bfloat16) for n in total]
    stack = serve.DecoderStack(serve.compressed_layers(words), HEADS, KV, D, 3, n_pages=30, page_size=16, max_len=160, int8=int8,
                               rotation=df11.rotation(D, base=500000.0), window=window, sinks=sinks,
                               head_norms=[tuple(w.cuda() for w in ws) for ws in weights] if norms else None)
    got, at = [[] for _ in xs], [0, 0, 0]
    for new in passes:
        rows = torch.cat([x[a:a + n] for x, a, n in zip(xs, at, new)]).to("cuda")
        out = (stack.token(rows) if new == [1, 1, 1] else stack.prompt(rows, new)).float().cpu()
        for s, part in enumerate(out.split(new)):
            got[s].append(part)
        at = [a + n for a, n in zip(at, new)]
    assert stack.lens == total
    # About 13 roundings to BF16 a layer lie on the way to an output, each at
    # most 2^-8 of what it rounds and independent of the others; 8-bit keys and
    # values are off by at most 1/254 of their row's largest, about 4 times the
    # row's root mean square: 2 x 4 / 254 more.
    bound = LAYERS * (13 * 2.0 ** -8 + (8 / 254 if int8 else 0))
    for x, parts in zip(xs, got):
        want = _plain(x.float(), layers, weights, window, sinks)
        off = (torch.cat(parts) - want).norm(dim=-1) / want.norm(dim=-1)
        assert float(off.max()) < bound, (float(off.max()), bound)


def test_a_window_without_a_rotation():
    """The stack's own rotary positions, with a window."""
    words = [[W.normal_bf16(s, seed=i, std=0.06) for i, s in enumerate(SHAPES)]]
    layers = [[torch.from_numpy(w.astype(np.uint32).view(np.int32) << 16).view(torch.float32) for w in ws] for ws in words]
    x = torch.randn(60, HIDDEN, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    stack = serve.DecoderStack(serve.compressed_layers(words), HEADS, KV, D, 1, n_pages=4, page_size=16, max_len=64, window=16, sinks=2)
    got = torch.cat([stack.prompt(x[:30].cuda(), [30]), stack.prompt(x[30:59].cuda(), [29]), stack.token(x[59:].cuda())]).float().cpu()
    want = _plain(x.float(), layers, None, 16, 2)
    off = (got - want).norm(dim=-1) / want.norm(dim=-1)
    assert float(off.max()) < 14 * 2.0 ** -8, float(off.max())


def test_stack_refuses_weights_without_a_rotation():
    words = [[W.normal_bf16(s, seed=i, std=0.06) for i, s in enumerate(SHAPES)]]
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(head_norms=[(w, w)]), dict(head_norms=[], rotation=df11.rotation(D)), dict(window=-1), dict(sinks=-1)):
        with pytest.raises(ValueError):
            serve.DecoderStack(serve.compressed_layers(words), HEADS, KV, D, 1, n_pages=2, page_size=16, max_len=32, **kw)


def test_the_command_runs(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["serve", "--layers", "1", "--prompts", "70,3", "--tokens", "2", "--window", "32", "--sinks", "2"])
    serve.main()
    out = capsys.readouterr().out
    assert out.count("finite True") == 4 and "finite False" not in out
