"""rotate_heads, kv_append, attend_chunk and windowed attend_token together, as
a layer uses them: on side streams, in captured graphs that are replayed, from
two host threads, and on buffers that change between replays, against the same
calls on the default stream."""
import threading

import pytest
import torch

import lossless_bf16_weight_amd as df11

import serve_chunk_util as CU
import serve_util as U
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
NEW, LENS, PS, H, HK, D = [20, 1, 77, 1], [3000, 800, 2477, 5], 16, 8, 2, 128


class _Layer:
    """A pass of a layer: new tokens appended, a chunk attended to, then a token in a window."""

    def __init__(self, seed, int8):
        t, n_pages = U.make_tables(LENS, PS, seed, width=300)
        k, v = CU.rand((n_pages, HK, PS, D), seed), CU.rand((n_pages, HK, PS, D), seed + 1)
        scales = [None, None]
        if int8:
            (k, ks), (v, vs) = ((x.to(DEV) for x in U.quantise32(x)) for x in (k, v))
            scales = [ks, vs]
        self.cache, self.pages = df11.KVCache(k, v, *scales), t.to(DEV)
        n = sum(NEW)
        at = torch.cat([torch.arange(m - a, m) for a, m in zip(NEW, LENS)])
        seq = torch.repeat_interleave(torch.arange(len(NEW)), torch.tensor(NEW))
        self.positions = at.to(torch.int32).to(DEV)
        self.slots = (t[seq, at // PS].long() * PS + at % PS).to(DEV)
        self.lens = torch.tensor(LENS, dtype=torch.int32, device=DEV)
        self.q_starts = U.starts_of(NEW).to(DEV)
        self.fused = CU.rand((n, H + 2 * HK, D), seed + 2)
        self.q, self.k, self.v = self.fused[:, :H], self.fused[:, H:H + HK], self.fused[:, H + HK:]
        self.rotation = df11.rotation(D, base=500000.0)
        self.w = CU.rand((D,), seed + 3)
        self.q1 = CU.rand((len(LENS), H, D), seed + 4)
        self.turned, self.out, self.out1 = (torch.empty(n, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(3))
        self.out1, self.q1_turned = torch.empty_like(self.q1), torch.empty_like(self.q1)
        self.at1 = (self.lens - 1).contiguous()
        assert df11.chunk_workspace(n, len(NEW), H, HK, D, PS, self.pages.shape[1]) > 0
        assert df11.token_workspace(len(LENS), H, HK, D, PS, self.pages.shape[1], 0, 2000, 4) > 0

    def go(self, stream=None):
        df11.kv_append(self.cache, self.k, self.v, self.positions, self.slots, self.rotation, k_weight=self.w, q=self.q, q_out=self.turned,
                       q_weight=self.w, stream=stream)
        df11.attend_chunk(self.turned, self.cache, self.pages, self.q_starts, self.lens, self.out, stream=stream)
        df11.rotate_heads(self.q1, None, self.at1, self.rotation, self.q1_turned, None, self.w, stream=stream)
        df11.attend_token(self.q1_turned, self.cache, self.pages, self.lens, self.out1, stream=stream, window=2000, sinks=4)

    def results(self):
        return [x.view(torch.int16).clone() for x in (self.turned, self.out, self.out1)]

    def forget(self):
        for x in (self.turned, self.out, self.out1, self.q1_turned):
            x.fill_(3.0)


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def _expected(c):
    c.go()
    torch.cuda.synchronize()
    got = c.results()
    U.within(c.out, *CU.chunk64(c.turned, c.cache, c.pages, NEW, LENS, D ** -0.5), "chunk")
    U.within(c.out1, *CU.chunk64(c.q1_turned, c.cache, c.pages, [1] * len(LENS), LENS, D ** -0.5, True, 2000, 4, weights=2.0 ** -14 * 1.01), "token")
    return got


@pytest.mark.parametrize("int8", [False, True])
def test_a_layer_on_side_streams(int8):
    log(f"a layer on side streams, int8 {int8}")
    both = [_Layer(101, int8), _Layer(151, int8)]
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
def test_a_layer_in_a_graph(int8):
    """Queries, lengths and starts change between replays; each replay equals
    the eager calls."""
    log(f"a layer in a graph, int8 {int8}")
    c = _Layer(201, int8)
    c.go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.go()
    for i in range(4):
        c.fused.copy_(CU.rand(c.fused.shape, 300 + i))
        c.q1.copy_(CU.rand(c.q1.shape, 400 + i))
        c.lens.copy_(torch.tensor([max(n, m - 700 * i) for n, m in zip(NEW, LENS)], dtype=torch.int32))
        c.q_starts.copy_(U.starts_of([20 + 10 * i, 1, 77 - 10 * i, 1]))
        c.forget()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = c.results()
        c.forget()
        c.go()
        torch.cuda.synchronize()
        assert _same(c.results(), replayed), i
        assert not bool((c.out == 3.0).all()) and not bool((c.out1 == 3.0).all())


def test_two_graphs_replayed_in_turn():
    """Two captured passes whose workspaces torch gave from one pool each."""
    both = [_Layer(301, False), _Layer(351, True)]
    want = [_expected(c) for c in both]
    graphs = []
    for c in both:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.go()
        graphs.append(g)
    for _ in range(3):
        for c in both:
            c.forget()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(_same(c.results(), w) for c, w in zip(both, want))


def test_two_host_threads():
    log("two host threads")
    both = [_Layer(501, False), _Layer(551, True)]
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


def test_the_binding_refuses_what_does_not_fit():
    """What the C ABI cannot see behind a pointer: shapes, types, devices."""
    c = _Layer(601, False)
    n = sum(NEW)
    good = dict(cache=c.cache, k=c.k, v=c.v, positions=c.positions, slots=c.slots, rotation=c.rotation, q=c.q, q_out=c.turned)
    for bad in (dict(k=c.k.float()), dict(v=c.v[:-1]), dict(positions=c.positions.long()), dict(positions=c.positions[:-1]),
                dict(positions=c.positions.cpu()), dict(slots=c.slots.int()), dict(slots=c.slots.cpu()), dict(q=c.q[..., :64]),
                dict(q_out=c.turned[:, :4]), dict(q_out=None), dict(k_out=c.turned), dict(q_weight=c.w[:64]), dict(k_weight=c.w.float()),
                dict(rotation=df11.rotation(D, device="cpu")), dict(rotation=df11.rotation(D, axes=[0] * 63 + [2]))):
        with pytest.raises(ValueError):
            df11.kv_append(**{**good, **bad})
    good = dict(q=c.turned, cache=c.cache, pages=c.pages, q_starts=c.q_starts, lens=c.lens, out=c.out)
    for bad in (dict(q=c.turned.float()), dict(pages=c.pages[:-1]), dict(q_starts=c.q_starts[:-1]), dict(lens=c.lens.long()), dict(out=c.out[:-1]),
                dict(out=c.out.cpu()), dict(window=-1), dict(sinks=-3), dict(workspace=torch.empty(8))):
        with pytest.raises(ValueError):
            df11.attend_chunk(**{**good, **bad})
    for bad in (dict(causal=False, window=5), dict(scale=0.0), dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(df11.DF11Error):
            df11.attend_chunk(**{**good, **bad})
    with pytest.raises(AttributeError):
        c.rotation.factor = 2.0
    assert n == c.out.shape[0]
