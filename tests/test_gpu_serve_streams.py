"""The calls that need a workspace, split kernels and joins among them, on side
streams, in a captured graph, and from two host threads at once, against the
same calls on the default stream."""
import threading

import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
LENS, Q_LENS, PS, H, HK, D, WIDTH = [3000, 1, 2477], [20, 1, 77], 16, 8, 2, 128, 400


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


class _Calls:
    """Inputs and outputs of both attentions, each of a size that is split."""

    def __init__(self, seed, int8):
        t, n_pages = U.make_tables(LENS, PS, seed, width=WIDTH)
        k, v = _rand((n_pages, HK, PS, D), seed), _rand((n_pages, HK, PS, D), seed + 1)
        scales = [None, None]
        if int8:
            (k, ks), (v, vs) = ((x.to(DEV) for x in U.quantise32(x)) for x in (k, v))
            scales = [ks, vs]
        self.cache, self.pages = df11.KVCache(k, v, *scales), t.to(DEV)
        self.lens = torch.tensor(LENS, dtype=torch.int32, device=DEV)
        self.q_starts, self.k_starts = U.starts_of(Q_LENS).to(DEV), U.starts_of(LENS).to(DEV)
        self.q, self.q1 = _rand((sum(Q_LENS), H, D), seed + 2), _rand((len(LENS), H, D), seed + 3)
        self.k, self.v = _rand((sum(LENS), HK, D), seed + 4), _rand((sum(LENS), HK, D), seed + 5)
        self.out, self.out1 = torch.empty_like(self.q), torch.empty_like(self.q1)
        assert df11.prompt_workspace(sum(Q_LENS), sum(LENS), len(LENS), H, HK, D) > 0
        assert df11.token_workspace(len(LENS), H, HK, D, PS, WIDTH) > 0

    def go(self, stream=None):
        df11.attend_prompt(self.q, self.k, self.v, self.q_starts, self.k_starts, self.out, stream=stream)
        df11.attend_token(self.q1, self.cache, self.pages, self.lens, self.out1, stream=stream)

    def results(self):
        return [x.view(torch.int16).clone() for x in (self.out, self.out1)]

    def forget(self):
        self.out.fill_(3.0)
        self.out1.fill_(3.0)


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def _expected(calls):
    calls.go()
    torch.cuda.synchronize()
    got = calls.results()
    U.within(calls.out, *U.prompt64(calls.q, calls.k, calls.v, Q_LENS, LENS, True, D ** -0.5), "prompt")
    U.within(calls.out1, *U.token64(calls.q1, calls.cache, calls.pages, LENS, D ** -0.5), "token")
    return got


@pytest.mark.parametrize("int8", [False, True])
def test_workspaces_on_side_streams(int8):
    """Two streams at work at once, each with workspaces of its own, which go
    back to the allocator while the kernels run."""
    log(f"workspaces on streams, int8 {int8}")
    both = [_Calls(101, int8), _Calls(151, int8)]
    want = [_expected(c) for c in both]
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(3):
        for c in both:
            c.forget()
        torch.cuda.synchronize()
        for _ in range(4):
            for c, s in zip(both, streams):
                c.go(s)
        torch.cuda.synchronize()
        assert all(_same(c.results(), w) for c, w in zip(both, want))


@pytest.mark.parametrize("int8", [False, True])
def test_workspaces_in_a_graph(int8):
    log(f"workspaces in a graph, int8 {int8}")
    calls = _Calls(201, int8)
    calls.go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls.go()
    for i in range(4):
        calls.q.copy_(_rand(calls.q.shape, 300 + i))
        calls.q1.copy_(_rand(calls.q1.shape, 400 + i))
        calls.lens.copy_(torch.tensor([n - 700 * i if n > 1 else n for n in LENS], dtype=torch.int32))
        calls.forget()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = calls.results()
        calls.forget()
        calls.go()
        torch.cuda.synchronize()
        assert _same(calls.results(), replayed), i
        assert not bool((calls.out1 == 3.0).all())


def test_two_host_threads():
    """Each thread's calls go to its own current stream."""
    log("two host threads")
    both = [_Calls(501, False), _Calls(551, True)]
    want = [_expected(c) for c in both]
    for c in both:
        c.forget()
    torch.cuda.synchronize()
    failed = []

    def work(c, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    c.go()
                torch.cuda.current_stream().synchronize()
            assert _same(c.results(), w)
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(both, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed and not any(t.is_alive() for t in threads), failed
