"""A decoder stack after passes that were refused, or that failed in a layer:
the same words as a stack that never saw them."""
import pytest
import torch

from lossless_bf16_weight_amd import serve
from lossless_bf16_weight_amd import workloads as W

from gpu_util import log
from test_gpu_serve_stack import D, HEADS, HIDDEN, KV, SHAPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
def test_refused_passes_leave_no_trace(int8):
    log(f"decoder stack after refused passes, int8 cache {int8}")
    words = [[W.normal_bf16(s, seed=10 * l + i, std=0.06) for i, s in enumerate(SHAPES)] for l in range(2)]
    loop = serve.compressed_layers(words)
    one, other = (serve.DecoderStack(loop, HEADS, KV, D, 2, n_pages=5, page_size=16, max_len=64, int8=int8) for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(90, HIDDEN, device="cuda", generator=gen).to(torch.bfloat16)
    refused = [lambda: one.prompt(x[:90], [20, 70]),                 # the second's table is too short
               lambda: one.prompt(x[:84], [60, 24]),                 # too few pages
               lambda: one.prompt(x[:30], [20, 9]),
               lambda: one.prompt(x[:20], [20]),
               lambda: one.prompt(x[:25].float(), [20, 5]),          # not BF16: a layer refuses it
               lambda: one.token(x[:2, :HIDDEN - 8])]                # a product does

    def refuse():
        for f in refused:
            with pytest.raises((ValueError, RuntimeError)):
                f()

    at = 0
    for new in ([20, 5], [3, 30], [1, 1], [1, 1]):
        refuse()
        rows = x[at:at + sum(new)]
        at += sum(new)
        got, want = ((s.token(rows) if new == [1, 1] else s.prompt(rows, new)) for s in (one, other))
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), new
        assert one.lens == other.lens and one.free == other.free


def test_a_prompt_of_no_tokens():
    """Rows that no sequence adds: an empty result, and nothing changes."""
    log("decoder stack, a prompt of no tokens")
    words = [[W.normal_bf16(s, seed=i, std=0.06) for i, s in enumerate(SHAPES)]]
    loop = serve.compressed_layers(words)
    one, other = (serve.DecoderStack(loop, HEADS, KV, D, 2, n_pages=4, page_size=16, max_len=32) for _ in range(2))
    x = torch.randn(9, HIDDEN, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)).to(torch.bfloat16)
    for new in ([3, 2], [0, 4]):
        assert one.prompt(x[:0], [0, 0]).shape == (0, HIDDEN)
        got, want = (s.prompt(x[:sum(new)], new) for s in (one, other))
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and one.lens == other.lens and one.free == other.free
