"""attend_token hands rows from lane to lane through a wave's own tile in LDS.
In the compiled kernels a step's writes of K, its reads, the writes of V and
its reads are apart: the compiler may move none past the barriers between
them, which cost no instruction."""
import re

from test_kernel_build import _compile

WRITE, READ = r"^\s*ds_write(?:2?_b64|_b128)", r"^\s*ds_read(?:2?_b64|_b128|_b64_tr_b\d+)"


def test_writes_and_reads_of_a_tile_are_apart(tmp_path):
    asm, _ = _compile("attend_token.hip", tmp_path)
    bodies = re.findall(r"^(\S*attend_token_kernel\S*):(.*?)^\s*\.section", asm, re.S | re.M)
    assert len(bodies) == 16
    for name, body in bodies:
        parts = re.split(r"^\s*; wave barrier.*$", body, flags=re.M)
        assert len(parts) >= 5, name
        parts[4] = re.split(r"^\s*s_barrier", parts[4], flags=re.M)[0]      # (the waves' join follows)
        kinds = [(len(re.findall(WRITE, p, re.M)), len(re.findall(READ, p, re.M))) for p in parts[1:5]]
        (k_written, a), (b, k_read), (v_written, c), (d, v_read) = kinds
        assert k_written and v_written and k_read and v_read and not (a or b or c or d), (name, kinds)
