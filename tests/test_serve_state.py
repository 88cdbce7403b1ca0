"""What a decoder stack (serve.py) holds of its sequences, on the CPU: a pass
that is refused, or fails in a layer, leaves lengths, free pages and page
tables as they were, and the next one is given the slots that it would have
been given."""
import pytest
import torch

from lossless_bf16_weight_amd import serve


class _Layers:
    """Stands for the layer loop: `fail` is what a pass raises."""
    fail = None

    def __len__(self):
        return 1

    def run(self, consumer):
        if self.fail:
            raise self.fail


def _stack(n_seqs=2, n_pages=3, max_len=64):
    return serve.DecoderStack(_Layers(), 2, 1, 64, n_seqs, n_pages=n_pages, page_size=16, max_len=max_len, device="cpu")


def _state(s):
    return list(s.lens), list(s.free), s.pages.clone()


def _same(a, b):
    return a[0] == b[0] and a[1] == b[1] and torch.equal(a[2], b[2])


def _rows(n):
    return torch.zeros(n, 8, dtype=torch.bfloat16)


@pytest.mark.parametrize("new,n_pages,max_len", [([20, 40], 3, 64),       # too few pages for the second
                                                 ([40, 20], 4, 64),
                                                 ([1, 33], 9, 32),        # the second's table is too short
                                                 ([16, 16], 1, 64)])
def test_a_pass_that_does_not_fit_changes_nothing(new, n_pages, max_len):
    s = _stack(2, n_pages, max_len)
    held = _state(s)
    with pytest.raises(RuntimeError):
        s._grow(new)
    assert _same(_state(s), held)
    with pytest.raises(RuntimeError):
        s.prompt(_rows(sum(new)), new)
    assert _same(_state(s), held)
    positions, slots = s._grow([3, 0])
    assert positions.tolist() == [0, 1, 2] and slots.tolist() == [0, 1, 2]


def test_a_token_that_does_not_fit_changes_nothing():
    s = _stack(2, 2)
    s._grow([5, 16])
    held = _state(s)
    with pytest.raises(RuntimeError):       # the second needs a third page
        s.token(_rows(2))
    assert _same(_state(s), held)


@pytest.mark.parametrize("rows,new", [(3, [2, 2]), (5, [2, 2]), (4, [4]), (4, [2, 1, 1]), (1, [2, -1])])
def test_counts_that_do_not_fit_the_rows_are_refused(rows, new):
    s = _stack()
    held = _state(s)
    with pytest.raises(ValueError):
        s.prompt(_rows(rows), new)
    assert _same(_state(s), held)


def test_a_token_of_other_than_one_row_a_sequence_is_refused():
    s = _stack()
    held = _state(s)
    for rows in (0, 1, 3):
        with pytest.raises(ValueError):
            s.token(_rows(rows))
    assert _same(_state(s), held)


@pytest.mark.parametrize("call", ["prompt", "token"])
def test_a_layer_that_fails_leaves_the_sequences_as_they_were(call):
    s = _stack()
    s._grow([16, 3])
    held = _state(s)
    s.loop.fail = ValueError("a layer")
    with pytest.raises(ValueError, match="a layer"):
        s.token(_rows(2)) if call == "token" else s.prompt(_rows(4), [3, 1])
    assert s.lens == held[0] and s.free == held[1] and torch.equal(s.pages[:, :1], held[2][:, :1])
    positions, slots = s._grow([1, 1])
    assert positions.tolist() == [16, 3] and slots.tolist() == [2 * 16, 1 * 16 + 3] and s.free == []


def test_growth_takes_pages_in_order():
    s = _stack(3, 6)
    positions, slots = s._grow([17, 0, 2])
    assert s.lens == [17, 0, 2] and s.free == [3, 4, 5] and s.pages[0, :2].tolist() == [0, 1] and int(s.pages[2, 0]) == 2
    assert positions.tolist() == [*range(17), 0, 1] and slots.tolist() == [*range(17), 32, 33]
    positions, slots = s._grow([1, 1, 15])
    assert positions.tolist() == [17, 0, *range(2, 17)] and slots.tolist() == [17, 48, *range(34, 48), 64]
    assert s.lens == [18, 1, 17] and s.free == [5]
