"""A decoder stack served from compressed weights: the layer loop decodes
layer l + 1 while layer l computes, with a paged key-value cache and the
attention operators beside the products (a small example of the parts
together; norms, rotary positions and the activation are plain torch).

    python -m lossless_bf16_weight_amd.serve [--layers N] [--prompts 500,37,1] [--tokens N] [--int8]

runs Llama-3-8B-shaped layers of synthetic weights: a prompt of each sequence,
a second piece behind it, then new tokens one at a time, and prints what each
pass takes."""
from __future__ import annotations

import argparse
import time
from typing import List, Sequence

import torch
import torch.nn.functional as F

from . import workloads
from ._lib import Plan, encode
from ._serve import attend_prompt, attend_token, kv_cache, kv_read, kv_write
from .jit import LayerLoop


def rotary(x: torch.Tensor, positions: torch.Tensor, base: float = 500000.0) -> torch.Tensor:
    """x [rows, heads, head_dim] turned by its rows' positions."""
    half = x.shape[-1] // 2
    angle = positions[:, None].float() * base ** (-torch.arange(half, device=x.device).float() / half)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat((a * c - b * s, b * c + a * s), -1).to(x.dtype)


def norm(x: torch.Tensor) -> torch.Tensor:
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-5)).to(x.dtype)


class DecoderStack:
    """Layers of the llama8b_block layout (q, k, v, o, gate, up, down) in a
    LayerLoop, with a cache of `n_pages` pages a layer for `n_seqs` sequences.
    Pages are handed out as sequences grow."""

    def __init__(self, loop: LayerLoop, n_heads: int, n_kv_heads: int, head_dim: int, n_seqs: int, n_pages: int,
                 page_size: int = 64, max_len: int = 8192, int8: bool = False, device: str = "cuda"):
        self.loop, self.heads, self.kv_heads, self.d, self.page_size = loop, n_heads, n_kv_heads, head_dim, page_size
        self.caches = [kv_cache(n_pages, n_kv_heads, page_size, head_dim, int8=int8, device=device) for _ in range(len(loop))]
        self.pages = torch.zeros(n_seqs, -(-max_len // page_size), dtype=torch.int32, device=device)
        self.lens: List[int] = [0] * n_seqs
        self.free = list(range(n_pages))
        self.device = device

    def _grow(self, new: Sequence[int]):
        """Makes room for new[s] tokens of each sequence; their positions and
        slots, and the new lengths.  Where they do not all fit, nothing changes."""
        if len(new) != len(self.lens) or min(new, default=0) < 0:
            raise ValueError(f"{list(new)}: a count for each of {len(self.lens)} sequences is needed")
        have = [-(-n // self.page_size) for n in self.lens]
        need = [-(-(a + n) // self.page_size) for a, n in zip(self.lens, new)]
        for s, n in enumerate(need):
            if n > self.pages.shape[1]:
                raise RuntimeError(f"sequence {s}: {self.lens[s] + new[s]} tokens are more than its page table holds")
        if sum(need) - sum(have) > len(self.free):
            raise RuntimeError(f"{sum(need) - sum(have)} pages are needed, {len(self.free)} are left")
        positions, slots = [], []
        for s, n in enumerate(new):
            if need[s] > have[s]:
                taken, self.free = self.free[:need[s] - have[s]], self.free[need[s] - have[s]:]
                self.pages[s, have[s]:need[s]] = torch.tensor(taken, dtype=torch.int32, device=self.device)
            at = torch.arange(self.lens[s], self.lens[s] + n, device=self.device)
            positions.append(at)
            slots.append(self.pages[s, at // self.page_size].long() * self.page_size + at % self.page_size)
            self.lens[s] += n
        return torch.cat(positions), torch.cat(slots)

    def _starts(self, lens: Sequence[int]) -> torch.Tensor:
        out = [0]
        for n in lens:
            out.append(out[-1] + n)
        return torch.tensor(out, dtype=torch.int32, device=self.device)

    def _run(self, x: torch.Tensor, new: Sequence[int], attend):
        """One pass of the stack over the next new[s] tokens of each sequence
        (rows of x); attend(layer, q, k, v) gives the attention.  A pass that
        fails leaves the lengths and pages as they were: what it had written
        lies past them."""
        if x.shape[0] != sum(new):
            raise ValueError(f"x: {x.shape[0]} rows for {sum(new)} tokens")
        held = list(self.lens), self.free
        state = [x]

        def layer(l: int, ws: List[torch.Tensor]):
            wq, wk, wv, wo, gate, up, down = ws
            x = state[0]
            h = norm(x)
            q, k, v = (F.linear(h, w).unflatten(1, (n, self.d)) for w, n in ((wq, self.heads), (wk, self.kv_heads), (wv, self.kv_heads)))
            q, k = rotary(q, positions), rotary(k, positions)
            kv_write(self.caches[l], k, v, slots)
            x = x + F.linear(attend(l, q, k, v).flatten(1), wo)
            h = norm(x)
            state[0] = x + F.linear(F.silu(F.linear(h, gate)) * F.linear(h, up), down)

        try:
            positions, slots = self._grow(new)
            self.loop.run(layer)
        except BaseException:
            self.lens, self.free = held
            raise
        return state[0]

    def prompt(self, x: torch.Tensor, new: Sequence[int]) -> torch.Tensor:
        """The next new[s] tokens of each sequence, rows of x packed in order
        (bfloat16): their hidden states after the last layer.  Sequences that
        have tokens in the cache attend to those too."""
        after = [a + n for a, n in zip(self.lens, new)]
        cached = any(self.lens)
        q_starts, k_starts = self._starts(new), self._starts(after)

        def attend(l, q, k, v):
            if cached:     # what came before is in the cache
                k, v = (torch.empty(sum(after), self.kv_heads, self.d, dtype=q.dtype, device=q.device) for _ in range(2))
                kv_read(self.caches[l], self.pages, k_starts, k, v)
            out = torch.empty_like(q)
            attend_prompt(q, k, v, q_starts, k_starts, out)
            return out

        return self._run(x, new, attend)

    def token(self, x: torch.Tensor) -> torch.Tensor:
        """One more token of every sequence (row s of x)."""
        lens = torch.tensor([n + 1 for n in self.lens], dtype=torch.int32, device=self.device)

        def attend(l, q, k, v):
            out = torch.empty_like(q)
            attend_token(q, self.caches[l], self.pages, lens, out)
            return out

        return self._run(x, [1] * len(self.lens), attend)


def compressed_layers(layers: Sequence[Sequence], device: str = "cuda") -> LayerLoop:
    """A LayerLoop over BF16 word arrays (one list of arrays a layer)."""
    containers = [[encode(w) for w in layer] for layer in layers]
    plans = [Plan(cs) for cs in containers]
    return LayerLoop(plans, [[torch.from_numpy(c).to(device) for c in cs] for cs in containers], device=device)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--prompts", default="500,37,1")
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--int8", action="store_true", help="keep the cache in 8 bits")
    args = ap.parse_args()
    new = [int(n) for n in args.prompts.split(",")]
    loop = compressed_layers([[s.make() for s in workloads.llama8b_block(l)] for l in range(args.layers)])
    most = 2 * max(new) + args.tokens
    stack = DecoderStack(loop, 32, 8, 128, len(new), n_pages=len(new) * (-(-most // 64)), max_len=most, int8=args.int8)
    gen = torch.Generator(device="cuda").manual_seed(0)

    def rows(n):
        return torch.randn(n, 4096, device="cuda", generator=gen).to(torch.bfloat16)

    def timed(what, f):
        torch.cuda.synchronize()
        t = time.perf_counter()
        out = f()
        torch.cuda.synchronize()
        print(f"{what}: {(time.perf_counter() - t) * 1e3:.2f} ms, lengths {stack.lens}, "
              f"finite {bool(torch.isfinite(out.float()).all())}", flush=True)

    timed("prompt", lambda: stack.prompt(rows(sum(new)), new))
    timed("second piece", lambda: stack.prompt(rows(sum(new)), new))
    for _ in range(args.tokens):
        timed("token", lambda: stack.token(rows(len(new))))


if __name__ == "__main__":
    main()
