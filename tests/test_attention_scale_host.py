"""spec_cache_attention refuses scales whose product is no 32-bit number, before any CUDA call (scores
of infinity times 0 would be NaN without a status bit)."""
import ctypes

import pytest

from speculative_decoding_draft_04_gb300 import _lib, build
from test_serving_host import EALIGN, EINVAL, make


@pytest.mark.parametrize("softmax_scale,k_scale,want", [
    (3e38, 1.0, EINVAL), (-3e38, 1.0, EINVAL), (1e21, 2.0 ** 60, EINVAL), (-1e21, 2.0 ** 60, EINVAL),
    # these are numbers: the next check answers (a misaligned table)
    (2e38, 1.0, EALIGN), (1e20, 2.0 ** 60, EALIGN), (3e38, 0.5, EALIGN), (0.0, 2.0 ** 60, EALIGN),
    (1e-38, 2.0 ** -60, EALIGN)])
def test_the_product_of_the_scales(softmax_scale, k_scale, want):
    build.build()
    a = make(_lib.CacheAttentionArgs, B=2, T=4, Hq=4, Hkv=2, D=64, dtype=1, page_size=16, num_pages=10, table_stride=5,
             mask_words=1, q_row_stride=256, q_head_stride=64, softmax_scale=softmax_scale, k_scale=k_scale,
             v_scale=1.0, workspace_bytes=1 << 40, block_table=0x100002)
    assert _lib.lib().spec_cache_attention(ctypes.byref(a), None) == want
