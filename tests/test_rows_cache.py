"""Which rows go past the last-level cache (rows_past_cache in csrc/rows.hip, called
as libmoe.so holds it; nothing is launched): by what a call can move, whatever the
buffer has room for."""
import ctypes

import pytest

import sparse_moe_layer_fp32_amd as moe


@pytest.fixture(scope="module")
def past_cache():
    f = moe.load_library()["_ZN3moe15rows_past_cacheEllil"]
    f.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    f.restype = ctypes.c_bool
    return f


@pytest.mark.parametrize("tokens,rows,top_k,row_bytes,past", [
    (8192, 65536, 8, 8192, True),        # every row is named
    (64, 65536, 8, 8192, False),         # 512 rows of a buffer of 537 MB
    (5, 1 << 26, 32, 128, False),
    (4097, 65536, 8, 8192, True),        # just above 256 MB of pairs
    (4096, 65536, 8, 8192, False),
    (32768, 1000, 8, 8192, False),       # fewer rows than pairs
    (8192, 65536, 8, 4096 + 128, True),  # codes and scales
    (64, 65536, 8, 4096 + 128, False),
    (1 << 25, 1 << 26, 32, 256, True), (0, 1 << 26, 1, 256, False), (1 << 25, 0, 1, 256, False)])
def test_rows_that_pairs_can_name(past_cache, tokens, rows, top_k, row_bytes, past):
    assert past_cache(tokens, rows, top_k, row_bytes) == past
