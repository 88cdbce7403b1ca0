"""Host side of rotate_heads, kv_append, attend_chunk and windows, on the CPU:
the argument structs that the binding packs are those of include/df11.h, the
refusals of the C ABI (all checks come before any device call), workspaces,
rotations, and the oracles of the GPU tests (a planted mistake is outside their
bounds)."""
import math
import os
import shutil
import struct
import subprocess

import pytest
import torch

import lossless_bf16_weight_amd as df11
from lossless_bf16_weight_amd import _serve as S

import serve_chunk_util as CU
import serve_heads_util as HU
import serve_util as U
from test_serve_host import CACHE, E_ARG, E_UNSUPPORTED, OK, ROOT, TABLE, P, _rows

TURN = ["rotation." + x for x in ("turns", "axes", "positions", "position_stride", "pairs", "n_axes", "flags", "factor")]
TOKEN = [*CACHE, *TABLE, *_rows("q"), *_rows("out"), "lens", "workspace", "workspace_bytes", "n_seqs", "n_heads", "scale", "reserved"]

STRUCTS = {
    "df11_rotate_heads_args": (S._HEADS, TURN + _rows("q") + _rows("k") + _rows("q_out") + _rows("k_out") +
                               ["q_weight", "k_weight", "n_tokens", "n_heads", "n_kv_heads", "head_dim", "eps"]),
    "df11_kv_append_args": (S._APPEND, CACHE + TURN + _rows("q") + _rows("k") + _rows("v") + _rows("q_out") + _rows("k_out") +
                            ["slots", "q_weight", "k_weight", "n_tokens", "n_heads", "eps"]),
    "df11_attend_token_window_args": (S._TOKEN_WINDOW, ["token." + x for x in TOKEN] + ["window", "sinks"]),
    "df11_attend_chunk_args": (S._CHUNK, CACHE + TABLE + _rows("q") + _rows("out") +
                               ["q_starts", "lens", "workspace", "workspace_bytes", "n_q", "n_seqs", "n_heads", "flags", "window", "sinks", "scale"]),
}


def test_packed_structs_are_those_of_the_header(tmp_path):
    if not shutil.which("gcc"):
        pytest.skip("gcc not available")
    lines = []
    for name, (_, fields) in STRUCTS.items():
        lines.append(f'printf("%zu", sizeof({name}));')
        lines += [f'printf(" %zu", offsetof({name}, {f}));' for f in fields]
        lines.append('printf("\\n");')
    c = tmp_path / "s.c"
    c.write_text('#include "df11.h"\n#include <stdio.h>\nint main(void) {' + "\n".join(lines) + "return 0; }\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROOT, "include"),
                    "-I/opt/rocm/include", str(c), "-o", str(exe)], check=True, capture_output=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    for line, (name, (packed, fields)) in zip(out, STRUCTS.items()):
        size, *offsets = map(int, line.split())
        codes = packed.format.lstrip("<")
        assert packed.size == size and len(codes) == len(fields), name
        assert [struct.calcsize("<" + codes[:i]) for i in range(len(codes))] == offsets, name


_TURN = [P, P, P, 3, 32, 3, 0, 1.0]
_CACHED, _TABLED = [P, P, 0, 0, 8, 16, 2, 128, 0, 0], [P, 4, 4, 0]
_Q, _K = [P, 512, 128], [P, 256, 128]
GOOD = {name: dict(zip(STRUCTS[name + "_args"][1], values)) for name, values in {
    "df11_rotate_heads": [*_TURN, *_Q, *_K, *_Q, *_K, P, P, 5, 4, 2, 128, 1e-6],
    "df11_kv_append": [*_CACHED, *_TURN, *_Q, *_K, *_K, *_Q, *_K, P, P, P, 5, 4, 1e-6],
    "df11_attend_token_window": [*_CACHED, *_TABLED, *_Q, *_Q, P, 0, 0, 2, 4, 0.1, 0, 10, 4],
    "df11_attend_chunk": [*_CACHED, *_TABLED, *_Q, *_Q, P, P, 0, 0, 5, 2, 4, 1, 10, 4, 0.1],
}.items()}

REFUSED = [
    ("cache.k", 0, E_ARG), ("cache.v", P + 8, E_ARG), ("cache.n_pages", 0, E_ARG), ("cache.page_size", 48, E_ARG), ("cache.head_dim", 96, E_UNSUPPORTED),
    ("cache.store", 2, E_ARG), ("cache.store", 1, E_ARG), ("cache.n_kv_heads", 0, E_ARG), ("cache.n_pages", 1 << 28, E_UNSUPPORTED),
    ("rotation.turns", 0, E_ARG), ("rotation.turns", P + 8, E_ARG), ("rotation.axes", P + 4, E_ARG), ("rotation.positions", 0, E_ARG),
    ("rotation.positions", P + 2, E_ARG), ("rotation.position_stride", -1, E_ARG), ("rotation.position_stride", 1 << 32, E_ARG),
    ("rotation.pairs", 12, E_ARG), ("rotation.pairs", 72, E_ARG), ("rotation.n_axes", 0, E_ARG), ("rotation.n_axes", 5, E_ARG),
    ("rotation.flags", 2, E_ARG), ("rotation.factor", float("nan"), E_ARG), ("rotation.factor", float("inf"), E_ARG),
    ("q.data", 0, E_ARG), ("q.data", P + 8, E_ARG), ("q.row_stride", -8, E_ARG), ("q.head_stride", 12, E_ARG), ("k.data", 0, E_ARG),
    ("k.row_stride", 4, E_ARG), ("v.data", P + 2, E_ARG), ("v.head_stride", 1 << 40, E_ARG), ("q_out.data", 0, E_ARG), ("q_out.row_stride", 0, E_ARG),
    ("q_out.head_stride", 64, E_ARG), ("k_out.row_stride", 128, E_ARG), ("k_out.data", P + 8, E_ARG), ("out.data", P + 8, E_ARG),
    ("out.row_stride", 0, E_ARG), ("out.head_stride", 64, E_ARG), ("q_weight", P + 2, E_ARG), ("k_weight", P + 8, E_ARG), ("eps", 0.0, E_ARG),
    ("eps", -1.0, E_ARG), ("eps", float("nan"), E_ARG), ("eps", float("inf"), E_ARG), ("slots", 0, E_ARG), ("slots", P + 4, E_ARG),
    ("n_tokens", 1 << 40, E_UNSUPPORTED), ("head_dim", 80, E_UNSUPPORTED), ("n_kv_heads", 1 << 16, E_ARG),
    ("table.pages", 0, E_ARG), ("table.pages", P + 2, E_ARG), ("table.row_stride", -1, E_ARG), ("table.width", 0, E_ARG),
    ("table.width", 1 << 26, E_UNSUPPORTED), ("lens", 0, E_ARG), ("lens", P + 2, E_ARG), ("q_starts", 0, E_ARG), ("q_starts", P + 1, E_ARG),
    ("scale", 0.0, E_ARG), ("scale", float("nan"), E_ARG), ("scale", 3e38, E_ARG), ("n_heads", 3, E_ARG), ("flags", 2, E_ARG),
    ("n_q", 1 << 33, E_UNSUPPORTED), ("n_q", (1 << 31) - 1, E_UNSUPPORTED), ("n_seqs", (1 << 32) - 1, E_UNSUPPORTED),
]
REFUSED += [("token." + f, v, s) for f, v, s in REFUSED]


def _call(name, fields):
    packed = STRUCTS[name + "_args"][0]
    codes = packed.format.lstrip("<")
    values = [float(v) if c == "f" else int(v) for c, v in zip(codes, fields.values())]
    return getattr(df11.lib(), name)(packed.pack(*values), 0, None)


@pytest.mark.parametrize("name", list(GOOD))
def test_refusals(name):
    n = 0
    good = GOOD[name]
    for field, value, status in REFUSED:
        if field not in good or (field == "n_heads" and "slots" in good):     # (any number of queries' heads may be appended)
            continue
        if field == "n_heads" and "head_dim" in good:
            continue
        got = _call(name, dict(good, **{field: value}))
        assert got == status, (name, field, value, got, df11.lib().df11_last_error())
        n += 1
    assert n >= 20
    assert getattr(df11.lib(), name)(None, 0, None) == E_ARG


def test_a_window_needs_the_causal_flag():
    assert _call("df11_attend_chunk", dict(GOOD["df11_attend_chunk"], flags=0)) == E_ARG


def test_calls_with_nothing_to_do_succeed():
    for name, field in (("df11_rotate_heads", "n_tokens"), ("df11_kv_append", "n_tokens"), ("df11_attend_chunk", "n_q"), ("df11_attend_chunk", "n_seqs"),
                        ("df11_attend_token_window", "token.n_seqs")):
        assert _call(name, dict(GOOD[name], **{field: 0})) == OK, (name, field)
    assert _call("df11_rotate_heads", dict(GOOD["df11_rotate_heads"], n_heads=0, n_kv_heads=0)) == OK
    assert _call("df11_attend_chunk", dict(GOOD["df11_attend_chunk"], n_q=0, lens=0, q_starts=0)) == OK


def test_too_many_waves_are_refused():
    assert _call("df11_rotate_heads", dict(GOOD["df11_rotate_heads"], n_tokens=(1 << 31) + 1)) == E_UNSUPPORTED
    assert _call("df11_rotate_heads", dict(GOOD["df11_rotate_heads"], n_tokens=(1 << 26) + 1)) == E_UNSUPPORTED


def test_workspaces():
    # a table of 256 positions is not split; a longer one is, and no further than the workgroups that run
    assert df11.chunk_workspace(64, 1, 32, 8, 128, 16, 16) == 0
    assert df11.chunk_workspace(64, 1000, 32, 8, 128, 16, 512) == 0
    need = df11.chunk_workspace(64, 1, 32, 8, 128, 16, 512)
    tile = 128 * 130 * 4
    most = 2 * 256 // 8 * 5 // 2 * 8 * tile + 16
    assert need and need % (8 * tile) == 16 and need <= most
    assert df11.chunk_workspace(64, 1, 32, 8, 128, 16, 1 << 20) == most
    assert df11.chunk_workspace(640, 2, 32, 8, 128, 16, 1 << 20) == most
    assert df11.chunk_workspace(640, 1, 32, 8, 128, 16, 1 << 20) == 3 * 256 * 2 * tile + 16      # (tiles of 256 rows)
    assert df11.chunk_workspace(64, 1, 32, 8, 128, 16, 1 << 20, 100, 4) == 0       # (a window of few steps)
    good = dict(GOOD["df11_attend_chunk"], **{"table.width": 4096, "window": 0})
    need = df11.chunk_workspace(5, 2, 4, 2, 128, 16, 4096)
    assert need
    for ws, size in ((0, 0), (P, need - 1), (P + 8, need)):
        assert _call("df11_attend_chunk", dict(good, workspace=ws, workspace_bytes=size)) == E_ARG
    # tokens: by the window, not by the table
    assert df11.token_workspace(1, 8, 2, 128, 16, 1 << 14) > df11.token_workspace(1, 8, 2, 128, 16, 1 << 14, 0, 4096, 4) > 0
    assert df11.token_workspace(1, 8, 2, 128, 16, 1 << 14, 0, 900, 4) == 0
    assert df11.token_workspace(1, 8, 2, 128, 16, 64, 0, 0, 4) == df11.token_workspace(1, 8, 2, 128, 16, 64)
    long_t = dict(GOOD["df11_attend_token_window"], **{"token.table.width": 4096, "window": 5000})
    need = df11.token_workspace(2, 4, 2, 128, 16, 4096, 0, 5000, 4)
    for ws, size in ((0, 0), (P, need - 1), (P + 8, need)):
        assert _call("df11_attend_token_window", dict(long_t, **{"token.workspace": ws, "token.workspace_bytes": size})) == E_ARG


def test_rotations():
    r = df11.rotation(64, base=500000.0, device="cpu")
    for i, t in enumerate(r.turns.tolist()):
        assert abs((t % 2 ** 64) / 2 ** 64 - 500000.0 ** (-i / 32) / (2 * math.pi)) < 2.0 ** -53
    assert r.axes is None and r.n_axes == 1 and not r.interleaved and r.factor == 1.0
    r = df11.rotation(32, freqs=[-1.0, 7.0] * 8, axes=[0, 1, 2, 0] * 4, interleaved=True, factor=0.5, device="cpu")
    turns = [(t % 2 ** 64) / 2 ** 64 for t in r.turns.tolist()]
    assert abs(turns[0] - (1 - 1 / (2 * math.pi))) < 2.0 ** -50 and abs(turns[1] - (7 / (2 * math.pi) - 1)) < 2.0 ** -50
    assert r.n_axes == 3 and r.axes.tolist() == [0, 1, 2, 0] * 4 and r.interleaved and r.factor == 0.5
    assert df11.rotation(0, device="cpu").turns.shape[0] == 0
    for bad in (dict(rotary_dim=24), dict(rotary_dim=-16), dict(rotary_dim=16, freqs=[1.0] * 7), dict(rotary_dim=16, axes=[0] * 7),
                dict(rotary_dim=16, axes=[4] * 8), dict(rotary_dim=16, axes=[-1] * 8), dict(rotary_dim=16, freqs=[math.inf] * 8),
                dict(rotary_dim=16, factor=math.nan)):
        with pytest.raises(ValueError):
            df11.rotation(device="cpu", **bad)


def test_the_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        df11.rotate_heads(x, None, None, None, x, None)
    with pytest.raises(ValueError):
        df11.rotate_heads(None, None, None, None, None, None)
    with pytest.raises(ValueError):
        df11.kv_append(df11.kv_cache(1, 2, 16, 64, device="cpu"), x, x, None, torch.zeros(3, dtype=torch.int64), None)
    with pytest.raises(ValueError):
        df11.attend_chunk(x, df11.kv_cache(1, 2, 16, 64, device="cpu"), None, None, torch.zeros(1, dtype=torch.int32), x)


# ---------------------------------------------------------------- the oracles

def _rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def test_heads_oracle_is_the_textbook_form():
    """Against complex numbers, and norms by hand."""
    x, w = _rand((4, 3, 64), 1), _rand((64,), 2)
    pos = torch.tensor([[0], [1], [77], [-5]], dtype=torch.int32)
    f = HU.freqs64(64, 10000.0)
    for neighbours in (False, True):
        y, _ = HU.heads64(x, pos, f, [0] * 32, neighbours, 1.5, w, 1e-6)
        z = x.double() / (x.double().pow(2).sum(-1, keepdim=True) / 64 + 1e-6).sqrt() * w.double()
        a, b = (z[..., 0::2], z[..., 1::2]) if neighbours else (z[..., :32], z[..., 32:])
        t = pos.double()[:, :, None] * torch.tensor(f, dtype=torch.float64)
        r = torch.complex(a, b) * torch.polar(torch.full_like(t, 1.5), t)
        got = (y[..., 0::2], y[..., 1::2]) if neighbours else (y[..., :32], y[..., 32:])
        assert torch.allclose(got[0], r.real, atol=1e-9) and torch.allclose(got[1], r.imag, atol=1e-9)


@pytest.mark.parametrize("plant", ["sign", "frequency", "position", "pairs", "weight", "eps", "axis"])
def test_heads_bounds_catch_a_planted_mistake(plant):
    x, w = _rand((6, 2, 64), 3), _rand((64,), 4)
    pos = torch.arange(1, 13, dtype=torch.int32).view(6, 2)
    f, axes = HU.freqs64(64, 10000.0), [0, 1] * 16
    y, err = HU.heads64(x, pos, f, axes, False, 1.0, w)
    U.within(y.to(torch.bfloat16), y, HU.bound_of(y, err), "the right result")
    wrong = {"sign": lambda: HU.heads64(x, -pos, f, axes, False, 1.0, w),
             "frequency": lambda: HU.heads64(x, pos, [v * 1.02 for v in f], axes, False, 1.0, w),
             "position": lambda: HU.heads64(x, pos + 1, f, axes, False, 1.0, w),
             "pairs": lambda: HU.heads64(x, pos, f, axes, True, 1.0, w),
             "weight": lambda: HU.heads64(x, pos, f, axes, False, 1.0, w.flip(0)),
             "eps": lambda: HU.heads64(x, pos, f, axes, False, 1.0, w, 0.02),
             "axis": lambda: HU.heads64(x, pos, f, axes[::-1], False, 1.0, w)}[plant]()[0]
    with pytest.raises(AssertionError):
        U.within(wrong.to(torch.bfloat16), y, HU.bound_of(y, err), plant)


@pytest.mark.parametrize("plant", ["window", "sinks", "position", "dropped key"])
def test_chunk_bounds_catch_a_planted_mistake(plant):
    q, k, v = (_rand((40, 64), 5 + i).double() for i in range(3))
    seen = CU.seen64(40, 40, True, 12, 3)
    out, bound = CU.attend64(q, k, v, seen, 0.125)
    U.within(out.to(torch.bfloat16), out, bound, "the right result")
    other = {"window": CU.seen64(40, 40, True, 11, 3), "sinks": CU.seen64(40, 40, True, 12, 4), "position": CU.seen64(40, 40, True, 12, 3).roll(1, 0),
             "dropped key": seen & (torch.arange(40) != 20)}[plant]
    with pytest.raises(AssertionError):
        U.within(CU.attend64(q, k, v, other, 0.125)[0].to(torch.bfloat16), out, bound, plant)


def test_chunk_oracle_is_the_one_of_prompts_and_tokens():
    lens, new = [37, 50, 8], [37, 5, 1]
    c = CU.Cached(lens, 2, 64, 16, False, seed=9, poison=False, device="cpu")
    q = _rand((sum(new), 4, 64), 10)
    out, _ = CU.chunk64(q, c.cache, c.table, new, lens, 0.125)
    rows = [torch.cat([U.gathered(x, None, c.table[s], m) for s, m in enumerate(lens)]) for x in c.cache[:2]]
    want, _ = U.prompt64(q, *rows, new, lens, True, 0.125)
    assert torch.allclose(out, want, atol=1e-12)
    last = torch.tensor([36, 41, 42])
    out, _ = CU.chunk64(q[last], c.cache, c.table, [1, 1, 1], lens, 0.125)
    want, _ = U.token64(q[last], c.cache, c.table, lens, 0.125)
    assert torch.allclose(out, want, atol=1e-12)
