"""spec_cache_attention's largest calls: a request's rows, rounded up to whole tiles of 128, stay 32-bit
numbers, and what would pass them is refused before any CUDA call."""
import ctypes

import pytest

from speculative_decoding_draft_04_gb300 import _lib, build
from test_serving_host import EALIGN, EINVAL, make

MOST = 2 ** 31 - 256


@pytest.mark.parametrize("T,Hq,want", [
    (16647160, 129, EINVAL), (2 ** 23 - 1, 256, EALIGN), (2 ** 23, 256, EINVAL), (MOST // 129, 129, EALIGN),
    (MOST // 129 + 1, 129, EINVAL), (MOST // 255, 255, EALIGN), (MOST // 255 + 1, 255, EINVAL),
    (2 ** 24 - 1, 127, EALIGN)])
def test_rows_of_a_request(T, Hq, want):
    build.build()
    assert want == EINVAL or T * Hq + 127 < 2 ** 31      # one key-value head: tiles of one request's rows
    a = make(_lib.CacheAttentionArgs, B=1, T=T, Hq=Hq, Hkv=1, D=64, dtype=1, page_size=16, num_pages=10, table_stride=5,
             mask_words=1, q_row_stride=256, q_head_stride=64, softmax_scale=0.1, k_scale=1.0, v_scale=1.0,
             workspace_bytes=1 << 40, block_table=0x100002)
    assert _lib.lib().spec_cache_attention(ctypes.byref(a), None) == want
