"""What a decoder stack (serve.py) hands to the operators and makes for them, on
the CPU with the operators replaced by recorders."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from lossless_bf16_weight_amd import serve

HEADS, KV, D, HIDDEN, PAGE = 2, 1, 64, 128, 16


class _Layers:
    """Stands for the layer loop: one layer of weights on the CPU."""

    def __len__(self):
        return 1

    def run(self, consumer):
        g = torch.Generator().manual_seed(1)
        shapes = [(HEADS * D, HIDDEN), (KV * D, HIDDEN), (KV * D, HIDDEN), (HIDDEN, HEADS * D), (32, HIDDEN), (32, HIDDEN), (HIDDEN, 32)]
        consumer(0, [torch.randn(s, generator=g).to(torch.bfloat16) for s in shapes])


class _Made(TorchDispatchMode):
    """Counts casts of int64 to int32."""
    casts = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        kwargs = kwargs or {}
        if func is torch.ops.aten._to_copy.default and args[0].dtype is torch.int64 and kwargs.get("dtype") is torch.int32:
            self.casts += 1
        return func(*args, **kwargs)


@pytest.fixture
def calls(monkeypatch):
    """The operators' calls of a pass as (name, args, keywords), and the tensors
    made of host data."""
    log, made = [], []
    for name in ("kv_write", "kv_append", "kv_read", "attend_prompt", "attend_chunk", "attend_token"):
        monkeypatch.setattr(serve, name, lambda *args, _name=name, **kw: log.append((_name, args, kw)))
    real = torch.tensor
    monkeypatch.setattr(torch, "tensor", lambda data, **kw: made.append(data) or real(data, **kw))
    return log, made


def _stack(rotation, window, max_len=512, n_seqs=2):
    r = serve.make_rotation(D, device="cpu") if rotation else None
    return serve.DecoderStack(_Layers(), HEADS, KV, D, n_seqs, n_pages=64, page_size=PAGE, max_len=max_len, device="cpu", rotation=r, window=window)


def _rows(n):
    return torch.zeros(n, HIDDEN, dtype=torch.bfloat16)


@pytest.mark.parametrize("rotation,window", [(False, 0), (True, 0), (True, 8), (False, 8)])
def test_a_pass_makes_what_it_uses(rotation, window, calls):
    """Indexes of host data, each a copy to the device: a prompt's starts, and
    either the starts of its keys or its lengths; a token's lengths.  32-bit
    positions where a rotation reads them."""
    log, made = calls
    s = _stack(rotation, window)
    s.prompt(_rows(5), [3, 2])
    s.prompt(_rows(4), [0, 4])
    s.token(_rows(2))
    made.clear()
    with _Made() as mode:
        s.prompt(_rows(3), [1, 2])
        assert made == [[0, 1, 3], [5, 9] if rotation or window else [0, 5, 14]]
        made.clear()
        s.token(_rows(2))
        assert made == [[6, 10]]
    assert mode.casts == (2 if rotation else 0)
    names = {name for name, _, _ in log}
    assert names == {"kv_append" if rotation else "kv_write", "attend_token"} | ({"attend_chunk"} if rotation or window else {"attend_prompt", "kv_read"})


@pytest.mark.parametrize("rotation,window", [(True, 0), (True, 8), (False, 8)])
def test_prompts_attend_over_the_entries_in_use(rotation, window, calls):
    """attend_chunk takes the table's width for the length of a single sequence:
    it is given the columns that the longest sequence uses, of the stack's own table."""
    log, _ = calls
    s = _stack(rotation, window, max_len=8192)
    after = [0, 0]
    for new in ([3, 2], [13, 0], [1, 40], [0, 0], [0, 100]):
        s.prompt(_rows(sum(new)), new)
        after = [a + n for a, n in zip(after, new)]
        name, args, _ = log[-1]
        pages, lens = args[2], args[4]
        assert name == "attend_chunk" and lens.tolist() == after
        assert pages.shape == (2, -(-max(after) // PAGE)) and pages.data_ptr() == s.pages.data_ptr() and pages.stride() == s.pages.stride()
        for i, n in enumerate(after):
            at = torch.arange(n)
            assert torch.equal(pages[i, at // PAGE], s.pages[i, at // PAGE])
    empty = _stack(rotation, window)
    empty.prompt(_rows(0), [0, 0])
    assert log[-1][1][2].shape == (2, 1)
    with pytest.raises(RuntimeError):      # (more than the table holds)
        empty.prompt(_rows(1000), [1000, 0])
