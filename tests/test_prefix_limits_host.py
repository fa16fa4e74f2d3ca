"""The limits of spec_prefix_attention's groups, as the header states them, before any CUDA call."""
import ctypes
import os
import re

import pytest

from speculative_decoding_draft_04_gb300 import _lib
from speculative_decoding_draft_04_gb300 import build as B
from tests.test_serving_host import EINVAL, make

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def call(groups, stride):
    """Without rows, so that what is allowed returns before it reads anything."""
    a = _lib.PrefixAttentionArgs(groups=groups, prefix_stride=stride, prefix_table=0x10000, prefix_len=0x20000,
                                 group_ptr=0x30000)
    a.own = make(_lib.CacheAttentionArgs, B=2, T=0, Hq=4, Hkv=2, D=64, dtype=1, page_size=16, num_pages=10,
                 table_stride=5, mask_words=1, q_row_stride=256, q_head_stride=64, softmax_scale=0.1, k_scale=1.0,
                 v_scale=1.0, workspace_bytes=1 << 40)
    return _lib.lib().spec_prefix_attention(ctypes.byref(a), None)


def test_the_header_says_what_is_refused():
    B.build()
    text = open(os.path.join(ROOT, "include", "spec.h")).read()
    m = re.search(r"(\d+) <= groups <= (\d+), prefix_stride >= (\d+), groups \* prefix_stride < 2\^31", text)
    least, most, stride = (int(x) for x in m.groups())
    allowed = [(least, stride), (most, stride), (2, 2 ** 30 - 1), (1, 2 ** 31 - 1)]
    refused = [(least - 1, stride), (most + 1, stride), (least, stride - 1), (2, 2 ** 30), (4096, 2 ** 19)]
    assert [call(*x) for x in allowed] == [0] * 4 and [call(*x) for x in refused] == [EINVAL] * 5
