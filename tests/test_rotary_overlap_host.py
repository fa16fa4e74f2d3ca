"""spec_rotary_append refuses a q_out whose rows or heads share addresses, before any CUDA call."""
import ctypes

import pytest

from speculative_decoding_draft_04_gb300 import _lib
from speculative_decoding_draft_04_gb300 import build as B
from tests.test_serving_host import EINVAL, make


def call(T, Hq, row, head):
    """EINVAL for overlapping strides; with the others the next refusal, of a CUDA device that is not there or of a
    missing cache, is another one."""
    a = make(_lib.RotaryAppendArgs, T=T, Hq=Hq, Hkv=2, D=64, R=64, dtype=1, page_size=16, num_pages=10, rope_rows=100,
             q_row_stride=512, q_head_stride=64, k_row_stride=512, k_head_stride=64, v_row_stride=512, v_head_stride=64,
             q_out_row_stride=row, q_out_head_stride=head, eps=1e-6, k_scale=1.0, v_scale=1.0)
    return _lib.lib().spec_rotary_append(ctypes.byref(a), None)


@pytest.mark.parametrize("T,Hq,row,head", [
    (4, 4, 256, 0), (4, 4, 0, 64), (4, 4, 0, 0), (4, 4, 248, 64), (4, 4, 256, 56), (4, 1, 56, 0), (1, 4, 0, 56),
    (4, 4, 64, 248), (4, 4, -248, 64), (4, 4, 64, 64), (4, 256, 2 ** 62, 2 ** 60)])
def test_overlapping_rows(T, Hq, row, head):
    B.build()
    assert call(T, Hq, row, head) == EINVAL


@pytest.mark.parametrize("T,Hq,row,head", [
    (4, 4, 256, 64), (4, 4, 512, 64), (4, 4, 64, 256), (4, 4, 72, 512), (4, 1, 64, 0), (1, 4, 0, 64), (1, 1, 0, 0),
    (4, 4, -256, 64), (4, 4, 256, -64), (4, 256, 2 ** 62, 2 ** 50)])
def test_rows_that_are_apart(T, Hq, row, head):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are none: only where no kernel can run")
    B.build()
    assert call(T, Hq, row, head) not in (0, EINVAL)
