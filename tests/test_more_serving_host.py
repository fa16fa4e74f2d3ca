"""Sampling, norm with rotation and append, attention with shared prefixes, on the host: the binding's
structs against the header, the refusals of the host-side checks before any CUDA call, and the
oracle's definitions against worked cases (no GPU needed)."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import serving as S
from speculative_decoding_draft_04_gb300 import _lib
from speculative_decoding_draft_04_gb300 import build as B
from tests.test_serving_host import EALIGN, EINVAL, EUNSUPPORTED, EWORKSPACE, make, refused

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MIRRORS = {"spec_prefix_attention_args": _lib.PrefixAttentionArgs, "spec_rotary_append_args": _lib.RotaryAppendArgs,
           "spec_sample_args": _lib.SampleArgs}


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


def fields(py):
    for f, t in py._fields_:
        yield from ((f"{f}.{g}" for g in fields(t)) if hasattr(t, "_fields_") else (f,))


def value(a, name):
    for part in name.split("."):
        a = getattr(a, part)
    return a


@pytest.mark.parametrize("py,fmt", [(_lib.PrefixAttentionArgs, _lib._PREFIX), (_lib.RotaryAppendArgs, _lib._ROTARY),
                                    (_lib.SampleArgs, _lib._SAMPLE)])
def test_packed_arguments_have_the_structs_layout(py, fmt):
    names = list(fields(py))
    packed = fmt.pack(*(i + 1 for i in range(len(names))))
    assert len(packed) == ctypes.sizeof(py)
    a = py.from_buffer_copy(packed)
    assert [value(a, f) for f in names] == [i + 1 for i in range(len(names))]


def test_sample_refusals(L):
    def base():
        return make(_lib.SampleArgs, B=2, n=3, V=100, dtype=1, b_stride=300, row_stride=100)
    refused(L.spec_sample, base, [({f: None}, EINVAL) for f in ("logits", "u", "tokens", "dev_status")] + [
        (dict(B=0), EINVAL), (dict(n=0), EINVAL), (dict(B=2 ** 20, n=2), EINVAL), (dict(V=0), EINVAL),
        (dict(V=1 << 24), EINVAL), (dict(dtype=2), EUNSUPPORTED), (dict(logits=0x100001), EALIGN),
        (dict(dtype=0, logits=0x100002), EALIGN),
        (dict(u=0x100002), EALIGN), (dict(top_p=0x100001), EALIGN), (dict(kept=0x100002), EALIGN)])


def test_rotary_append_refusals(L):
    def base():
        return make(_lib.RotaryAppendArgs, T=4, Hq=4, Hkv=2, D=64, R=64, dtype=1, page_size=16, num_pages=10,
                    rope_rows=100, q_row_stride=512, q_head_stride=64, k_row_stride=512, k_head_stride=64,
                    v_row_stride=512, v_head_stride=64, q_out_row_stride=256, q_out_head_stride=64, eps=1e-6,
                    k_scale=1.0, v_scale=1.0)
    q = base().q
    refused(L.spec_rotary_append, base, [({f: None}, EINVAL) for f in (
        "q", "k", "v", "positions", "slots", "rope", "q_out", "cache", "dev_status")] + [
        (dict(T=-1), EINVAL), (dict(T=1 << 24), EINVAL), (dict(Hq=0), EINVAL), (dict(Hq=257), EINVAL),
        (dict(Hkv=0), EINVAL), (dict(Hkv=257), EINVAL), (dict(num_pages=2 ** 28), EINVAL), (dict(rope_rows=0), EINVAL),
        (dict(k_scale=0.0), EINVAL), (dict(v_scale=float("nan")), EINVAL), (dict(eps=-1e-6), EINVAL),
        (dict(eps=float("inf")), EINVAL), (dict(eps=float("nan")), EINVAL),
        (dict(T=(1 << 24) - 1, Hq=256, D=256, R=256), EINVAL),
        (dict(D=96), EUNSUPPORTED), (dict(dtype=3), EUNSUPPORTED), (dict(page_size=8), EUNSUPPORTED),
        (dict(R=0), EUNSUPPORTED), (dict(R=16), EUNSUPPORTED), (dict(R=48), EUNSUPPORTED), (dict(R=96), EUNSUPPORTED),
        (dict(q=0x100008), EALIGN), (dict(rope=0x100008), EALIGN), (dict(q_weight=0x100008), EALIGN),
        (dict(positions=0x100002), EALIGN), (dict(q_row_stride=508), EALIGN), (dict(q_out_head_stride=60), EALIGN),
        (dict(q_out=q), EINVAL), (dict(q_out=q, q_out_row_stride=512, q_out_head_stride=128), EINVAL)])


def test_prefix_attention_refusals(L):
    def base():
        a = _lib.PrefixAttentionArgs(groups=2, prefix_stride=3, prefix_table=0x10000, prefix_len=0x20000,
                                     group_ptr=0x30000)
        a.own = make(_lib.CacheAttentionArgs, B=2, T=4, Hq=4, Hkv=2, D=64, dtype=1, page_size=16, num_pages=10,
                     table_stride=5, mask_words=1, q_row_stride=256, q_head_stride=64, softmax_scale=0.1,
                     k_scale=1.0, v_scale=1.0, workspace_bytes=1 << 40)
        return a
    refused(L.spec_prefix_attention, base, [({f: None}, EINVAL) for f in ("prefix_table", "prefix_len", "group_ptr")] + [
        (dict(groups=0), EINVAL), (dict(groups=4097), EINVAL), (dict(prefix_stride=0), EINVAL),
        (dict(groups=4096, prefix_stride=2 ** 20), EINVAL), (dict(prefix_len=0x20002), EALIGN)])
    for change, want in [(dict(q=None), EINVAL), (dict(B=0), EINVAL), (dict(Hq=5), EINVAL), (dict(D=80), EUNSUPPORTED),
                         (dict(out=0x100008), EALIGN), (dict(workspace=None), EWORKSPACE),
                         (dict(workspace_bytes=_lib.spec_cache_attention_workspace_bytes(4, 2, 64)), EWORKSPACE),
                         (dict(workspace=0x100008), EALIGN)]:
        a = base()
        for k, v in change.items():
            setattr(a.own, k, v)
        assert L.spec_prefix_attention(ctypes.byref(a), None) == want, change
    size = _lib.spec_prefix_attention_workspace_bytes
    assert size(100, 32, 8, 128) >= _lib.spec_cache_attention_workspace_bytes(32, 8, 128) + 100 * 32 * (4 * 128 + 8)
    for args in [(-1, 32, 8, 128), (1 << 24, 32, 8, 128), (2 ** 23, 256, 8, 128), (4, 8, 3, 128), (4, 8, 8, 72)]:
        assert size(*args) == 0, args


def test_the_binding_checks_types_and_shapes():
    torch = pytest.importorskip("torch")
    i32, u8 = torch.int32, torch.uint8
    x, st = torch.zeros((4, 2, 64)), torch.zeros(4, dtype=i32)
    cache = torch.zeros((3, 2, 1, 18 * 64), dtype=u8)
    rope = torch.zeros((8, 32, 2))
    for bad in [dict(q=x[:3]), dict(q=x[0]), dict(q=x[..., :32]), dict(k=x[:, :1]), dict(v=x.to(torch.bfloat16)),
                dict(rope=rope[..., 0]), dict(rope=rope[..., :1]), dict(q_out=x.to(torch.bfloat16)), dict(k=x[0]),
                dict(cache=cache[0]), dict(eps="1"), dict(k_scale=1e300), dict(q=x)]:       # the last: not on a GPU
        a = dict(q=x, k=x, v=x, positions=st, slots=st, rope=rope, q_out=x, cache=cache, dev_status=st)
        a.update(bad)
        with pytest.raises(_lib.SpecError):
            _lib.spec_rotary_append(**a)
    for bad in [dict(logits=x[0]), dict(u=x), dict(logits=x)]:
        a = dict(logits=x, u=x[..., 0], tokens=st.view(4, 1), dev_status=st)
        a.update(bad)
        with pytest.raises(_lib.SpecError):
            _lib.spec_sample(**a)
    for table in (st, st.view(1, 2, 2), st.view(2, 2)):
        with pytest.raises(_lib.SpecError):
            _lib.spec_prefix_attention(x, cache, st.view(2, 2), st[:2], st[:3], table, st[:2], st[:3], x, st, st, 1.0)


# ------------------------------------------------------------- the oracle

def test_sampling_by_hand():
    x = np.log([0.1, 0.4, 0.1, 0.3, 0.1])
    assert [S.sample(x, 1.0, u)[0] for u in (0.0, 0.0999, 0.1001, 0.55, 0.85, 0.95)] == [0, 0, 1, 2, 3, 4]
    token, lp, kept, _ = S.sample(x, 1.0, 0.5, top_k=2)            # 0.4 and 0.3
    assert (token, kept) == (1, 2) and abs(lp - math.log(4 / 7)) < 1e-12
    assert S.sample(x, 1.0, 0.6, top_k=2)[0] == 3
    assert S.sample(x, 1.0, 0.5, top_p=0.69)[2] == 2               # 0.4 alone is less, with 0.3 it is more
    assert S.sample(x, 1.0, 0.5, top_p=0.71)[2] == 3               # the first of the three equal ones
    assert S.sample(x, 1.0, 0.99, top_p=0.71)[0] == 3
    assert S.sample(x, 1.0, 0.5, min_p=0.7)[2] == 2 and S.sample(x, 1.0, 0.5, min_p=0.8)[2] == 1
    assert S.sample(x, 1.0, 0.5, top_k=4, top_p=0.99)[2] == 4      # of the mass of four
    assert S.sample(x, 0.5, 0.5, min_p=0.5)[2] == 2                # (3/4)^2 = 0.5625
    assert S.sample(np.array([-np.inf, 0.0, -np.inf]), 1.0, 0.9, top_k=2)[:3] == (1, 0.0, 1)
    assert S.sample(np.array([-np.inf, -np.inf]), 1.0, 0.5) is None and S.sample(np.array([0.0, np.nan]), 1.0, 0.5) is None


def test_sampling_follows_the_distribution():
    rng = np.random.default_rng(0)
    x = rng.normal(size=12)
    p = np.exp(x / 0.7) / np.exp(x / 0.7).sum()
    grid = (np.arange(20000) + 0.5) / 20000
    n = np.bincount([S.sample(x, 0.7, u)[0] for u in grid], minlength=12)
    assert np.abs(n / 20000 - p).max() <= 1e-4


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, a = rng.normal(size=(5, 2, 64)), rng.normal(size=(5, 16)) * 100
    rows = np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)
    y = S.rotated(x, rows, interleaved=interleaved)
    i = np.arange(16)
    re, im = (2 * i, 2 * i + 1) if interleaved else (i, i + 16)
    z = (x[..., re] + 1j * x[..., im]) * np.exp(1j * a)[:, None]
    # coordinates up to 5 in fp32: two products and a sum, 3 half ulps of 8 and the table's rounding
    assert np.abs(y[..., re] - z.real).max() < 2e-6 and np.abs(y[..., im] - z.imag).max() < 2e-6
    assert np.array_equal(y[..., 32:], x[..., 32:].astype(np.float32))
    w = rng.normal(size=64).astype(np.float32)
    y = S.rotated(x, rows, weight=w, interleaved=interleaved)
    want = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6) * w
    assert np.abs(y[..., 32:] - want[..., 32:]).max() < 2e-6
