"""Host side of the serving operators, on the CPU: the argument structs that
the binding packs are those of include/df11.h, the refusals of the C ABI (all
checks come before any device call), the workspace sizes, and the oracle of
the GPU tests (a planted mistake is outside its bounds)."""
import os
import shutil
import struct
import subprocess

import pytest
import torch

import lossless_bf16_weight_amd as df11
from lossless_bf16_weight_amd import _serve as S

import serve_util as U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, E_ARG, E_UNSUPPORTED = 0, 1, 3

# fields of the C structs in the order that the binding packs them
CACHE = ["cache.k", "cache.v", "cache.k_scale", "cache.v_scale", "cache.n_pages", "cache.page_size", "cache.n_kv_heads",
         "cache.head_dim", "cache.store", "cache.reserved"]
TABLE = ["table.pages", "table.row_stride", "table.width", "table.reserved"]


def _rows(x):
    return [f"{x}.data", f"{x}.row_stride", f"{x}.head_stride"]


STRUCTS = {
    "df11_kv_write_args": (S._WRITE, CACHE + _rows("k") + _rows("v") + ["slots", "n_tokens"]),
    "df11_kv_read_args": (S._READ, CACHE + TABLE + _rows("k") + _rows("v") + ["starts", "n_tokens", "n_seqs", "reserved"]),
    "df11_attend_token_args": (S._TOKEN, CACHE + TABLE + _rows("q") + _rows("out") +
                               ["lens", "workspace", "workspace_bytes", "n_seqs", "n_heads", "scale", "reserved"]),
    "df11_attend_prompt_args": (S._PROMPT, _rows("q") + _rows("k") + _rows("v") + _rows("out") +
                                ["q_starts", "k_starts", "workspace", "workspace_bytes", "n_q", "n_k", "n_seqs", "n_heads",
                                 "n_kv_heads", "head_dim", "flags", "scale"]),
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


P = 1 << 20      # an aligned address that is never read: every call here is refused or has nothing to do

GOOD = {
    "df11_kv_write": dict(zip(STRUCTS["df11_kv_write_args"][1], [P, P, 0, 0, 8, 16, 2, 128, 0, 0, P, 256, 128, P, 256, 128, P, 5])),
    "df11_kv_read": dict(zip(STRUCTS["df11_kv_read_args"][1], [P, P, 0, 0, 8, 16, 2, 128, 0, 0, P, 4, 4, 0, P, 256, 128, P, 256, 128,
                                                               P, 5, 2, 0])),
    "df11_attend_token": dict(zip(STRUCTS["df11_attend_token_args"][1], [P, P, 0, 0, 8, 16, 2, 128, 0, 0, P, 4, 4, 0, P, 512, 128,
                                                                         P, 512, 128, P, 0, 0, 2, 4, 0.1, 0])),
    "df11_attend_prompt": dict(zip(STRUCTS["df11_attend_prompt_args"][1], [P, 512, 128, P, 256, 128, P, 256, 128, P, 512, 128, P, P,
                                                                           0, 0, 5, 5, 1, 4, 2, 128, 1, 0.1])),
}

REFUSED = [
    ("cache.k", 0, E_ARG), ("cache.v", P + 8, E_ARG), ("cache.n_pages", 0, E_ARG), ("cache.page_size", 8, E_ARG),
    ("cache.page_size", 48, E_ARG), ("cache.page_size", 2048, E_ARG), ("cache.head_dim", 96, E_UNSUPPORTED),
    ("cache.head_dim", 0, E_UNSUPPORTED), ("cache.store", 2, E_ARG), ("cache.store", 1, E_ARG),     # (8 bits without scales)
    ("cache.n_kv_heads", 0, E_ARG), ("cache.n_pages", 1 << 28, E_UNSUPPORTED),
    ("k.data", 0, E_ARG), ("k.data", P + 2, E_ARG), ("k.row_stride", 4, E_ARG), ("k.row_stride", -8, E_ARG), ("v.head_stride", 1 << 40, E_ARG),
    ("q.data", 0, E_ARG), ("q.head_stride", 12, E_ARG), ("out.data", P + 8, E_ARG), ("out.row_stride", 0, E_ARG), ("out.head_stride", 64, E_ARG),
    ("slots", 0, E_ARG), ("slots", P + 4, E_ARG), ("n_tokens", 1 << 40, E_UNSUPPORTED), ("starts", 0, E_ARG), ("starts", P + 2, E_ARG),
    ("table.pages", 0, E_ARG), ("table.pages", P + 2, E_ARG), ("table.row_stride", -1, E_ARG), ("table.width", 0, E_ARG),
    ("table.width", 1 << 26, E_UNSUPPORTED), ("lens", 0, E_ARG), ("scale", 0.0, E_ARG), ("scale", -1.0, E_ARG),
    ("scale", 3e38, E_ARG), ("scale", float("nan"), E_ARG), ("scale", float("inf"), E_ARG), ("n_heads", 3, E_ARG), ("n_heads", 0, E_ARG),
    ("n_kv_heads", 0, E_ARG), ("head_dim", 80, E_UNSUPPORTED), ("flags", 2, E_ARG), ("n_q", 1 << 33, E_UNSUPPORTED),
    ("n_k", 1 << 33, E_UNSUPPORTED), ("q_starts", 0, E_ARG), ("k_starts", P + 1, E_ARG), ("n_seqs", (1 << 32) - 1, E_UNSUPPORTED),
]


def _call(name, fields):
    packed = STRUCTS[name + "_args"][0]
    codes = packed.format.lstrip("<")
    # (negative values of unsigned fields do not occur)
    values = [float(v) if c == "f" else int(v) for c, v in zip(codes, fields.values())]
    return getattr(df11.lib(), name)(packed.pack(*values), 0, None)


@pytest.mark.parametrize("name", list(GOOD))
def test_refusals(name):
    n = 0
    for field, value, status in REFUSED:
        if field not in GOOD[name]:
            continue
        got = _call(name, dict(GOOD[name], **{field: value}))
        assert got == status, (name, field, value, got, df11.lib().df11_last_error())
        assert df11.lib().df11_last_error()
        n += 1
    assert n >= 10
    assert getattr(df11.lib(), name)(None, 0, None) == E_ARG


def test_key_rows_too_far_apart_are_refused():
    for x in ("k", "v"):
        assert _call("df11_attend_prompt", dict(GOOD["df11_attend_prompt"], **{f"{x}.row_stride": 1 << 24})) == E_UNSUPPORTED


def test_reads_of_more_waves_than_a_launch_holds_are_refused():
    for heads, n, seqs in ((65535, 1 << 15, 2), (2, 1 << 30, 2), (8, 5, (1 << 24) - 1)):
        assert _call("df11_kv_read", dict(GOOD["df11_kv_read"], **{"cache.n_kv_heads": heads, "n_tokens": n, "n_seqs": seqs})) == E_UNSUPPORTED


def test_output_rows_that_overlap_are_refused():
    # (inputs may overlap; a single row or head has no stride)
    for name, what, other in (("df11_kv_read", "v", "n_tokens"), ("df11_attend_token", "out", "n_seqs"), ("df11_attend_prompt", "out", "n_q")):
        for row, head in ((128, 128), (512, 120), (0, 0), (256, 128 if name != "df11_kv_read" else 256)):
            assert _call(name, dict(GOOD[name], **{f"{what}.row_stride": row, f"{what}.head_stride": head})) == E_ARG, (name, row, head)


def test_calls_with_nothing_to_do_succeed():
    assert _call("df11_kv_write", dict(GOOD["df11_kv_write"], n_tokens=0)) == OK
    assert _call("df11_kv_read", dict(GOOD["df11_kv_read"], n_tokens=0)) == OK
    assert _call("df11_kv_read", dict(GOOD["df11_kv_read"], n_seqs=0)) == OK
    assert _call("df11_attend_token", dict(GOOD["df11_attend_token"], n_seqs=0)) == OK
    assert _call("df11_attend_prompt", dict(GOOD["df11_attend_prompt"], n_seqs=0)) == OK
    assert _call("df11_attend_prompt", dict(GOOD["df11_attend_prompt"], n_q=0)) == OK


def test_workspace_sizes():
    assert df11.token_workspace(1, 8, 2, 128, 16, 64) == 0               # 1024 positions: taken whole
    parts = df11.token_workspace(1, 8, 2, 128, 16, 65) // (8 * 130 * 4)
    assert parts > 1 and df11.token_workspace(1, 8, 2, 128, 16, 65) == parts * 8 * 130 * 4
    assert df11.token_workspace(3, 8, 2, 64, 16, 4096) % (3 * 8 * 66 * 4) == 0
    assert df11.token_workspace(1, 8, 3, 128, 16, 64) == 0               # (refused by the call itself)
    assert df11.prompt_workspace(4096, 4096, 1, 32, 8, 128) == 0
    need = df11.prompt_workspace(4, 4096, 1, 8, 2, 64)
    assert need and need % (2 * 128 * 66 * 4) == 0         # (whole tiles of 128 rows of each kv head)
    # too little, none, and misaligned
    long_q = dict(GOOD["df11_attend_prompt"], n_q=4, n_k=8192)
    need = df11.prompt_workspace(4, 8192, 1, 4, 2, 128)
    for ws, size in ((0, 0), (P, need - 1), (P + 8, need)):
        assert _call("df11_attend_prompt", dict(long_q, workspace=ws, workspace_bytes=size)) == E_ARG
    long_t = dict(GOOD["df11_attend_token"], **{"table.width": 4096})
    need = df11.token_workspace(2, 4, 2, 128, 16, 4096)
    for ws, size in ((0, 0), (P, need - 1), (P + 8, need)):
        assert _call("df11_attend_token", dict(long_t, workspace=ws, workspace_bytes=size)) == E_ARG


def test_every_page_size_starts_ranges_with_a_page():
    """Parts are whole numbers of pages, whatever the page size: the bytes of
    the workspace give their number, and they cover the table."""
    for page in (16, 32, 64, 128, 256, 512, 1024):
        for width in (1, 2, 3, 5, 17, 100, 1000):
            for seqs in (1, 3, 40, 500):
                need = df11.token_workspace(seqs, 4, 2, 64, page, width)
                parts = need // (seqs * 4 * 66 * 4) if need else 1
                assert parts <= max(1, -(-width * page // 128)), (page, width, seqs)
                # the longest part is at most 1280 positions, or a page or two
                assert parts >= width * page / max(1280, 2 * page), (page, width, seqs)


@pytest.mark.parametrize("plant", ["mask", "scale", "swap", "dropped key"])
def test_oracle_bounds_catch_a_planted_mistake(plant):
    """A wrong mask, scale, order of values or a key left out, rounded to BF16,
    is outside the bounds of the right result."""
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(40, 1, 64, generator=g).to(torch.bfloat16) for _ in range(3))
    out, bound = U.prompt64(q, k, v, [40], [40], True, 0.125)
    U.within(out.to(torch.bfloat16), out, bound, "the right result")
    if plant == "mask":
        wrong, _ = U.prompt64(q, k, v, [40], [40], False, 0.125)
    elif plant == "scale":
        wrong, _ = U.prompt64(q, k, v, [40], [40], True, 0.12)
    elif plant == "swap":
        v = v.clone()
        v[[3, 4]] = v[[4, 3]]
        wrong, _ = U.prompt64(q, k, v, [40], [40], True, 0.125)
    else:
        q64, k64, v64 = (x[:, 0].double() for x in (q, k, v))
        wrong = U.attend64(q64, k64, v64, [min(i + 1, 39) for i in range(40)], 0.125)[0][:, None]
    with pytest.raises(AssertionError):
        U.within(wrong.to(torch.bfloat16), out, bound, plant)
