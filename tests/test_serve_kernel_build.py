"""Properties of the compiled serving kernels that their speed and safety
depend on and that a small change can lose without any test failing: no
scratch, no flat memory instructions, no packed 32-bit arithmetic, the waves a
SIMD that their registers were fitted for, and prompt attention's loads in
flight over a whole step."""
import re

import pytest

from test_kernel_build import _compile, _remark


@pytest.mark.parametrize("src", ["kv_cache.hip", "attend_token.hip", "attend_prompt.hip"])
def test_no_scratch_flat_or_packed_arithmetic(src, tmp_path):
    asm, remarks = _compile(src, tmp_path)
    assert all(v == 0 for v in _remark(remarks, r"ScratchSize \[bytes/lane\]")), src
    assert not re.findall(r"^\s*flat_(?:load|store|atomic)\w*", asm, re.M)
    assert not re.findall(r"^\s*v_pk_(?:add|mul|fma)_f32", asm, re.M)


def _occupancy(remarks, name):
    blocks = re.split(r"Function Name: ", remarks)[1:]
    found = [int(re.search(r"Occupancy \[waves/SIMD\]: (\d+)", b).group(1)) for b in blocks if name in b.split()[0]]
    assert found, name
    return found


def test_waves_a_simd(tmp_path):
    _, remarks = _compile("attend_prompt.hip", tmp_path)
    assert all(v >= 2 for v in _occupancy(remarks, "attend_prompt_kernel"))
    _, remarks = _compile("attend_token.hip", tmp_path)
    assert all(v >= 3 for v in _occupancy(remarks, "attend_token_kernel"))


def test_prompt_products_do_not_wait_for_memory(tmp_path):
    """The next step's loads into LDS stay in flight: no block of matrix
    instructions waits for vector memory."""
    asm, _ = _compile("attend_prompt.hip", tmp_path)
    bodies = re.findall(r"^(\S*attend_prompt_kernel\S*):(.*?)^\s*\.section", asm, re.S | re.M)
    assert len(bodies) == 4
    for name, body in bodies:
        assert "buffer_load_dwordx4" in body and " lds" in body, name
        blocks = [b for b in re.split(r"^\.LBB\S+:", body, flags=re.M) if b.count("v_mfma") >= 4]
        assert blocks, name
        for b in blocks:
            assert not re.search(r"s_waitcnt [^\n]*vmcnt", b), name
