"""No output of fdllm_decode_attention may lie over any input, the RoPE tables
included (addresses are stand-ins that nothing reads)."""
import ctypes

import pytest

from kv_cache_attention_flash_b200 import _lib

MB = 1 << 26
NAMES = ["q", "k", "v", "positions", "slots", "rope_cos", "rope_sin", "k_pool", "v_pool", "block_table", "seq_lens",
         "starts", "out", "lse", "workspace"]
SHAPE = dict(batch=2, n_heads=4, n_kv_heads=2, head_dim=64, n_layers=2, num_pages=8, page_size=16,
             max_blocks_per_seq=4, max_position=100, dtype=0, in_dtype=0, out_dtype=1, scale=0.125, q_stride=256,
             k_stride=128, v_stride=128)


@pytest.mark.parametrize("put", ["out", "lse", "workspace", "k_pool", "v_pool"])
@pytest.mark.parametrize("over", [n for n in NAMES if n not in ("k_pool", "v_pool", "out", "lse", "workspace")])
def test_an_output_over_an_input_is_refused(put, over):
    lib = _lib.load()
    at = {n: (i + 1) * MB for i, n in enumerate(NAMES)}
    at[put] = at[over]
    d = _lib.Decode(*[SHAPE[n] for n, _ in _lib.Decode._fields_])
    r = lib.fdllm_decode_attention(ctypes.byref(d), 0, *[at[n] for n in NAMES], 1 << 30, None, None)
    assert r == _lib.FDLLM_ERR_INVALID_ARG and b"overlaps" in lib.fdllm_last_error()
    if over.startswith("rope"):                  # the last bytes of the table: 100 x 32 doubles
        at[put] = at[over] + 100 * 32 * 8 - 16
        r = lib.fdllm_decode_attention(ctypes.byref(d), 0, *[at[n] for n in NAMES], 1 << 30, None, None)
        assert r == _lib.FDLLM_ERR_INVALID_ARG and b"overlaps" in lib.fdllm_last_error()
