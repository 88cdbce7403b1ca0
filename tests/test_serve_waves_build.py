"""Waves a SIMD of the serving kernels as the division of their work counts on
them (serve.cpp): eight of heads.hip's, and of attend_chunk's workgroups as many
as it takes to run at a time, two a compute unit, with heads of 64 three (a
workgroup of four waves has one on each SIMD)."""
import re

import pytest

from test_kernel_build import _compile
from test_serve_kernel_build import _occupancy

LDS = 160 * 1024


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    return {src: _compile(src, tmp_path_factory.mktemp("asm")) for src in ("heads.hip", "attend_chunk.hip")}


def _lds(asm, kernel):
    """Bytes of LDS of each kernel whose name holds `kernel`."""
    return {name: int(n) for name, n in re.findall(r"^\s*\.amdhsa_kernel (\S+)\s*\n\s*\.amdhsa_group_segment_fixed_size (\d+)", asm, re.M) if kernel in name}


def test_heads_have_eight_waves(compiled):
    asm, remarks = compiled["heads.hip"]
    assert _occupancy(remarks, "heads_kernel") == [8] * 12
    assert all(n * 8 <= LDS for n in _lds(asm, "heads_kernel").values())      # (four waves a workgroup)


@pytest.mark.parametrize("d,at_a_time", [(64, 3), (128, 2)])
def test_chunks_have_the_workgroups_that_are_planned(d, at_a_time, compiled):
    asm, remarks = compiled["attend_chunk.hip"]
    waves = _occupancy(remarks, f"attend_chunk_kernelILi{d}ELb")
    assert len(waves) == 8
    four = [w for kernel in ("0ELb0", "0ELb1", "1ELb0", "1ELb1") for w in _occupancy(remarks, f"attend_chunk_kernelILi{d}ELb{kernel}ELj4E")]
    assert len(four) == 4 and all(w >= at_a_time for w in four)
    eight = [w for kernel in ("0ELb0", "0ELb1", "1ELb0", "1ELb1") for w in _occupancy(remarks, f"attend_chunk_kernelILi{d}ELb{kernel}ELj8E")]
    assert len(eight) == 4 and all(w >= 2 for w in eight)                     # (one workgroup, two waves a SIMD)
    lds = {n: b for n, b in _lds(asm, f"attend_chunk_kernelILi{d}E").items() if "Lj4E" in n}
    assert len(lds) == 4 and all(b * at_a_time <= LDS for b in lds.values())
