"""Properties of the compiled kernels of heads.hip and attend_chunk.hip that
their speed and safety depend on (as test_serve_kernel_build.py for the others):
no scratch, no flat memory instructions, no packed 32-bit arithmetic, the waves
a SIMD that their registers were fitted for, and loads in flight over a step."""
import re

import pytest

from test_kernel_build import _compile, _remark
from test_serve_handover import READ, WRITE
from test_serve_kernel_build import _occupancy


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    return {src: _compile(src, tmp_path_factory.mktemp("asm")) for src in ("heads.hip", "attend_chunk.hip", "attend_token.hip")}


@pytest.mark.parametrize("src", ["heads.hip", "attend_chunk.hip"])
def test_no_scratch_flat_or_packed_arithmetic(src, compiled):
    asm, remarks = compiled[src]
    assert all(v == 0 for v in _remark(remarks, r"ScratchSize \[bytes/lane\]")), src
    assert not re.findall(r"^\s*flat_(?:load|store|atomic)\w*", asm, re.M)
    assert not re.findall(r"^\s*v_pk_(?:add|mul|fma)_f32", asm, re.M)


def test_waves_a_simd(compiled):
    assert all(v >= 4 for v in _occupancy(compiled["heads.hip"][1], "heads_kernel"))
    assert all(v >= 2 for v in _occupancy(compiled["attend_chunk.hip"][1], "attend_chunk_kernel"))
    assert all(v >= 3 for v in _occupancy(compiled["attend_token.hip"][1], "attend_window_kernel"))


def test_writes_and_reads_of_a_wave_s_tile_are_apart(compiled):
    """As test_serve_handover.py for attend_token: windows, and the chunk's
    sequences of one token."""
    found = re.findall(r"^(\S*attend_window_kernel\S*):(.*?)^\s*\.section", compiled["attend_token.hip"][0], re.S | re.M)
    assert len(found) == 16
    single = [(n, b) for n, b in re.findall(r"^(\S*attend_chunk_kernel\S*):(.*?)^\s*\.section", compiled["attend_chunk.hip"][0], re.S | re.M) if "Lj4E" in n]
    assert len(single) == 8
    for name, body in found + single:
        parts = re.split(r"^\s*; wave barrier.*$", body, flags=re.M)
        assert len(parts) >= 5, name
        parts[4] = re.split(r"^\s*s_barrier", parts[4], flags=re.M)[0]
        kinds = [(len(re.findall(WRITE, p, re.M)), len(re.findall(READ, p, re.M))) for p in parts[1:5]]
        (k_written, a), (b, k_read), (v_written, c), (d, v_read) = kinds
        assert k_written and v_written and k_read and v_read and not (a or b or c or d), (name, kinds)


def test_products_do_not_wait_for_memory(compiled):
    """The next step's loads stay in flight: no block of the tiles' matrix
    instructions waits for vector memory (but the careful pass, which loads in it)."""
    asm, _ = compiled["attend_chunk.hip"]
    bodies = re.findall(r"^(\S*attend_chunk_kernel\S*):(.*?)^\s*\.section", asm, re.S | re.M)
    assert len(bodies) == 16
    for name, body in bodies:
        words = "ELb0E" in name.split("attend_chunk_kernel")[1][:10]
        assert not words or ("buffer_load_dwordx4" in body and " lds" in body), name
        blocks = [b for b in re.split(r"^\.LBB\S+:", body, flags=re.M) if b.count("v_mfma_f32_32x32x16") >= 4 and not re.search(r"buffer_load[^\n]* lds", b)]
        assert len(blocks) >= 4, name
        for b in blocks:
            assert not re.search(r"s_waitcnt [^\n]*vmcnt", b), name
