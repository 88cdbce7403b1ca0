"""Calls that a launch cannot hold are refused on the host, before any device
call: a grid's x dimension times its workgroup's threads stays below 2^32, its
y and z dimensions within 65,535.  (Every call here is refused.)"""
import pytest

import lossless_bf16_weight_amd as df11

from test_serve_host import E_UNSUPPORTED, GOOD, _call


def _refused(name, **fields):
    return _call(name, dict(GOOD[name], **fields)) == E_UNSUPPORTED


@pytest.mark.parametrize("d,heads,tokens", [
    (128, 2, 1 << 29),                       # 2^33 threads
    (128, 2, (1 << 28) - 15),                # one token past 2^24 - 1 workgroups of 512 chunks of 16 bytes
    (128, 1, (1 << 29) - 31),
    (64, 2, (1 << 29) - 31),
    (64, 65535, 1 << 30),
    (128, 65535, (1 << 64) - 1),
])
def test_writes_of_more_threads_than_a_launch_holds(d, heads, tokens):
    rows = {f"{x}.{s}_stride": 0 for x in "kv" for s in ("row", "head")}
    assert _refused("df11_kv_write", **{"cache.head_dim": d, "cache.n_kv_heads": heads, "n_tokens": tokens, **rows})


def test_2_to_the_24_workgroups_of_256_threads_are_refused():
    # reads: a tile of 16 tokens of one head of 128 is one wave, four waves a workgroup
    one = {f"{x}.{s}_stride": v for x in "kv" for s, v in (("row", 128), ("head", 0))}
    assert _refused("df11_kv_read", **{"cache.n_kv_heads": 1, "n_tokens": ((1 << 26) - 2) * 16, "n_seqs": 2, **one})
    # a token: the join has a workgroup a query head
    assert _refused("df11_attend_token", **{"cache.n_kv_heads": 1, "n_heads": 16, "n_seqs": 1 << 20, "q.row_stride": 2048,
                                            "out.row_stride": 2048})
    # prompts: rows of a head and its sequences, in tiles of 128
    assert _refused("df11_attend_prompt", n_q=128 * ((1 << 24) - 2), n_seqs=2, n_heads=1, n_kv_heads=1, **{"out.row_stride": 128})


def test_prompt_sizes_whose_product_passes_64_bits():
    """2^32 + 65,536 tile slots of 2^32 - 65,535 kv heads are 2^64 + 65,536 workgroups."""
    kv, n_q = (1 << 32) - 65535, 128 * 65537
    strides = {"out.row_stride": 128, "out.head_stride": 128 * n_q}
    assert _refused("df11_attend_prompt", n_q=n_q, n_seqs=(1 << 32) - 1, n_heads=kv, n_kv_heads=kv, **strides)
    assert df11.prompt_workspace(n_q, 5, (1 << 32) - 1, kv, kv, 128) == 0
