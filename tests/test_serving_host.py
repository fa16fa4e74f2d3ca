"""The serving operators on the host: the binding's structs against the header, and every refusal
of the host-side checks before any CUDA call (no GPU needed)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from speculative_decoding_draft_04_gb300 import _lib
from speculative_decoding_draft_04_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MIRRORS = {"spec_block_tables_args": _lib.BlockTablesArgs, "spec_cache_append_args": _lib.CacheAppendArgs,
           "spec_cache_attention_args": _lib.CacheAttentionArgs, "spec_logprobs_args": _lib.LogprobsArgs}
EINVAL, EUNSUPPORTED, EALIGN, EWORKSPACE = -1, -2, -3, -4


@pytest.fixture(scope="module")
def L():
    B.build()
    return _lib.lib()


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "spec.h"', "int main(void) {"]
    for cname, py in MIRRORS.items():
        lines.append(f'  printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True, capture_output=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        cname, field, value = line.split()
        py = MIRRORS[cname]
        assert int(value) == (ctypes.sizeof(py) if field == "sizeof" else getattr(py, field).offset), line


@pytest.mark.parametrize("py,fmt", [(_lib.BlockTablesArgs, _lib._TABLES), (_lib.CacheAppendArgs, _lib._APPEND),
                                    (_lib.CacheAttentionArgs, _lib._ATTENTION), (_lib.LogprobsArgs, _lib._LOGPROBS)])
def test_packed_arguments_have_the_structs_layout(py, fmt):
    values = [i + 1 for i in range(len(py._fields_))]
    packed = fmt.pack(*values)
    assert len(packed) == ctypes.sizeof(py)
    a = py.from_buffer_copy(packed)
    assert [getattr(a, f) for f, _ in py._fields_] == values


def make(py, **kw):
    """Arguments whose pointers are distinct, aligned and non-NULL."""
    a = py()
    for i, (f, t) in enumerate(py._fields_):
        if t is ctypes.c_void_p:
            setattr(a, f, 0x100000 * (i + 1))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def refused(fn, base, cases):
    assert fn(None, None) == EINVAL
    for change, want in cases:
        a = base()
        for k, v in change.items():
            setattr(a, k, v)
        assert fn(ctypes.byref(a), None) == want, change


def test_block_tables_refusals(L):
    def base():
        return make(_lib.BlockTablesArgs, B=4, page_size=16, num_pages=100, table_stride=10, max_rows=50)
    null = [({f: None}, EINVAL) for f in ("seq_len", "new_len", "num_blocks", "ring_pos", "free_ring",
                                          "block_table", "seq_len_out", "kv_len", "num_blocks_out",
                                          "ring_pos_out", "row_ptr", "slots", "positions", "dev_status")]
    same = base()
    refused(L.spec_block_tables, base, null + [
        (dict(B=0), EINVAL), (dict(B=4097), EINVAL), (dict(num_pages=0), EINVAL), (dict(table_stride=0), EINVAL),
        (dict(max_rows=0), EINVAL), (dict(max_rows=2 ** 31 - 1), EINVAL),
        (dict(B=4096, table_stride=2 ** 20), EINVAL), (dict(num_pages=2 ** 28), EINVAL),
        (dict(page_size=24), EUNSUPPORTED), (dict(page_size=256), EUNSUPPORTED),
        (dict(seq_len_out=same.seq_len), EINVAL), (dict(num_blocks_out=same.num_blocks), EINVAL),
        (dict(ring_pos_out=same.ring_pos), EINVAL), (dict(kv_len=same.accept_len), EINVAL),
        (dict(slots=0x100004), EALIGN), (dict(positions=0x100008), EALIGN), (dict(ring_pos=0x100004), EALIGN),
        (dict(seq_len=0x100002), EALIGN)])


def test_cache_append_refusals(L):
    def base():
        return make(_lib.CacheAppendArgs, T=4, Hkv=2, D=64, dtype=1, page_size=16, num_pages=10, k_row_stride=128,
                    k_head_stride=64, v_row_stride=128, v_head_stride=64, k_scale=1.0, v_scale=1.0)
    refused(L.spec_cache_append, base, [({f: None}, EINVAL) for f in ("k", "v", "slots", "cache", "dev_status")] + [
        (dict(T=-1), EINVAL), (dict(T=1 << 24), EINVAL), (dict(Hkv=0), EINVAL), (dict(Hkv=257), EINVAL),
        (dict(num_pages=0), EINVAL), (dict(num_pages=2 ** 28), EINVAL),
        (dict(k_scale=0.0), EINVAL), (dict(v_scale=-1.0), EINVAL), (dict(k_scale=float("nan")), EINVAL),
        (dict(k_scale=float("inf")), EINVAL), (dict(v_scale=2.0 ** -61), EINVAL),
        (dict(D=96), EUNSUPPORTED), (dict(D=512), EUNSUPPORTED), (dict(dtype=2), EUNSUPPORTED),
        (dict(page_size=8), EUNSUPPORTED), (dict(k=0x100008), EALIGN), (dict(cache=0x100008), EALIGN),
        (dict(k_row_stride=132), EALIGN), (dict(v_head_stride=68), EALIGN), (dict(v_stored=0x100008), EALIGN),
        (dict(dtype=0, k_row_stride=130), EALIGN), (dict(T=(1 << 24) - 1, Hkv=256, D=256), EINVAL)])


def test_cache_attention_refusals(L):
    def base():
        return make(_lib.CacheAttentionArgs, B=2, T=4, Hq=4, Hkv=2, D=64, dtype=1, page_size=16, num_pages=10,
                    table_stride=5, mask_words=1, q_row_stride=256, q_head_stride=64, softmax_scale=0.1,
                    k_scale=1.0, v_scale=1.0, workspace_bytes=1 << 40)
    refused(L.spec_cache_attention, base, [({f: None}, EINVAL) for f in (
        "q", "cache", "block_table", "kv_len", "row_ptr", "out", "dev_status")] + [
        (dict(B=0), EINVAL), (dict(B=4097), EINVAL), (dict(T=-1), EINVAL), (dict(Hkv=0), EINVAL),
        (dict(Hq=5), EINVAL), (dict(Hq=1), EINVAL), (dict(Hq=258), EINVAL), (dict(num_pages=0), EINVAL),
        (dict(table_stride=0), EINVAL), (dict(table_stride=2 ** 30), EINVAL), (dict(mask_words=0), EINVAL),
        (dict(softmax_scale=float("nan")), EINVAL), (dict(softmax_scale=float("inf")), EINVAL),
        (dict(k_scale=0.0), EINVAL), (dict(v_scale=float("nan")), EINVAL),
        (dict(D=80), EUNSUPPORTED), (dict(dtype=-1), EUNSUPPORTED), (dict(page_size=48), EUNSUPPORTED),
        (dict(q=0x100004), EALIGN), (dict(out=0x100008), EALIGN), (dict(q_row_stride=252), EALIGN),
        (dict(workspace=None), EWORKSPACE), (dict(workspace_bytes=16), EWORKSPACE),
        (dict(workspace=0x100008), EALIGN)])
    assert _lib.spec_cache_attention_workspace_bytes(32, 8, 128) > 0
    for args in [(8, 3, 128), (4, 8, 128), (300, 1, 64), (8, 0, 64), (8, 8, 72)]:
        assert _lib.spec_cache_attention_workspace_bytes(*args) == 0, args


def test_logprobs_refusals(L):
    def base():
        return make(_lib.LogprobsArgs, B=2, n=3, V=100, K=5, dtype=1, b_stride=300, row_stride=100,
                    workspace_bytes=1 << 40)
    refused(L.spec_logprobs, base, [({f: None}, EINVAL) for f in (
        "logits", "tokens", "logprob", "entropy", "top_ids", "top_logprobs", "dev_status")] + [
        (dict(B=0), EINVAL), (dict(n=0), EINVAL), (dict(B=2 ** 20, n=2), EINVAL), (dict(V=0), EINVAL),
        (dict(V=1 << 24), EINVAL), (dict(K=-1), EINVAL), (dict(V=4), EINVAL), (dict(K=0), EINVAL),
        (dict(K=33), EUNSUPPORTED), (dict(dtype=5), EUNSUPPORTED), (dict(logits=0x100008), EALIGN),
        (dict(tokens=0x100002), EALIGN), (dict(workspace=None), EWORKSPACE), (dict(workspace_bytes=8), EWORKSPACE),
        (dict(workspace=0x100004), EALIGN)])
    assert _lib.spec_logprobs_workspace_bytes(8, 32000, 20) > 0
    for args in [(0, 100, 1), (2 ** 20 + 1, 100, 1), (4, 0, 0), (4, 2 ** 24, 1), (4, 100, 33), (4, 3, 4)]:
        assert _lib.spec_logprobs_workspace_bytes(*args) == 0, args


def test_cache_bytes(L):
    assert _lib.spec_cache_bytes(10, 8, 64, 128) == 10 * 8 * 4 * 18 * 128
    for args in [(0, 8, 64, 128), (10, 0, 64, 128), (10, 8, 63, 128), (10, 8, 64, 100), (2 ** 28, 8, 64, 128)]:
        assert _lib.spec_cache_bytes(*args) == 0, args


def test_the_binding_checks_types_and_shapes():
    torch = pytest.importorskip("torch")
    i32, u8 = torch.int32, torch.uint8
    x = torch.zeros((4, 2, 64))
    cache = torch.zeros((3, 2, 1, 18 * 64), dtype=u8)
    st, slots = torch.zeros(4, dtype=i32), torch.zeros(4, dtype=i32)
    for bad in [dict(k=x[:, :1]), dict(v=x.to(torch.bfloat16)), dict(cache=cache[..., :100]),
                dict(cache=cache.to(torch.int8)), dict(k=x.transpose(1, 2)), dict(k=x)]:   # the last: not on a GPU
        a = dict(k=x, v=x, slots=slots, cache=cache, dev_status=st)
        a.update(bad)
        with pytest.raises(_lib.SpecError):
            _lib.spec_cache_append(**a)
    with pytest.raises(_lib.SpecError):
        _lib.spec_logprobs(torch.zeros((1, 2, 8)), slots, st, st, st, st)
    with pytest.raises(_lib.SpecError):
        _lib.spec_cache_attention(x, cache, slots.view(2, 2), slots[:2], slots[:3], x, st, st, 1.0)
    with pytest.raises(_lib.SpecError):
        _lib.spec_block_tables(slots, None, slots.float(), slots, slots, slots, slots.view(2, 2), slots, slots,
                               slots, slots, slots, slots, slots, st, 16)
