"""Rotation and append, attention with shared prefixes and sampling where offsets pass 32 bits: the same
bits as for the same numbers near the start.  And their tensors and streams of another device, which are
refused before anything is enqueued (one GPU stands for two, as in test_binding_devices_gpu)."""
import types

import numpy as np
import pytest

from tests import serving as H

pytestmark = pytest.mark.gpu
HQ, HKV, D, PAGE = 16, 8, 128, 64


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_draft_04_gb300 import build as B
    B.build()
    return t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 9])
def test_a_cache_of_more_than_32_bits(torch, dtype, rows):
    L, rng, dt = H.lib(), np.random.default_rng(rows), H.storage(torch, dtype)
    near, far = 8, 65000
    page_bytes = HKV * PAGE // 16 * 18 * D
    assert (far - near) * page_bytes > 2 ** 32
    prefix, own = 150, 70                                    # pages 0 to 2, and 3 to 4 and 5 to 6 of two requests
    table = np.array([[3, 4], [5, 6]], np.int32)
    T = prefix + 2 * own
    qkv = H.dev(rng.normal(size=(T, HQ + 2 * HKV, D)), dt)
    a = rng.uniform(-1000, 1000, (200, D // 2))
    rope = H.dev(np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32))
    at = np.concatenate([np.arange(prefix), 3 * PAGE + np.arange(own), 5 * PAGE + np.arange(own)]).astype(np.int32)
    positions = np.concatenate([np.arange(prefix), np.arange(own), np.arange(own)]).astype(np.int32)
    query = H.dev(rng.normal(size=(2 * rows, HQ, D)), dt)
    got = []
    for pages in (near, far):
        shift = pages - near                                 # the last pages
        cache = torch.empty((pages, HKV, PAGE // 16, 18 * D), dtype=torch.uint8, device="cuda")
        cache[shift:] = 0
        q = qkv[:, :HQ].clone()
        st = H.new_status()
        L.spec_rotary_append(q, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], H.dev(positions), H.dev(at + shift * PAGE), rope,
                             q, cache, st, 0.011, 0.003)
        out = torch.empty_like(query)
        lse = torch.empty((2 * rows, HQ), device="cuda")
        ws = torch.empty(L.spec_prefix_attention_workspace_bytes(2 * rows, HQ, HKV, D), dtype=torch.uint8, device="cuda")
        L.spec_prefix_attention(query, cache, H.dev(table + shift), H.dev(np.array([own, own], np.int32)),
                                H.dev(np.array([0, rows, 2 * rows], np.int32)),
                                H.dev(np.array([[0, 1, 2]], np.int32) + shift), H.dev(np.array([prefix], np.int32)),
                                H.dev(np.array([0, 2], np.int32)), out, st, ws, D ** -0.5, 0.011, 0.003, lse=lse)
        torch.cuda.synchronize()
        assert H.status(st) == 0
        got.append((cache[shift:].clone(), q, out, lse))
        del cache
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert got[0][2].float().abs().sum() > 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_more_than_32_bits_apart(torch, dtype):
    L, rng, dt = H.lib(), np.random.default_rng(5), H.storage(torch, dtype)
    apart, V = 2 ** 31 + 8 if dtype == "bf16" else 2 ** 30 + 4, 40001
    space = torch.empty(2 * apart + V, dtype=dt, device="cuda")
    x = H.dev(rng.normal(size=(3, 1, V)) * 3, dt)
    wide = space.as_strided((3, 1, V), (apart, V, 1))
    wide.copy_(x)
    got = []
    for logits in (x, wide):
        tokens, kept = (torch.full((3, 1), 77, dtype=torch.int32, device="cuda") for _ in range(2))
        st = H.new_status()
        L.spec_sample(logits, H.dev(np.array([[0.1], [0.5], [0.9]], np.float32)), tokens, st,
                      top_p=H.dev(np.array([0.9, 1.0, 0.5], np.float32)), kept=kept)
        torch.cuda.synchronize()
        assert H.status(st) == 0
        got.append((tokens, kept))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    # queries, rotated in place
    q = H.dev(rng.normal(size=(3, 4, 64)), dt)
    wide = space.as_strided((3, 4, 64), (apart, 64, 1))
    wide.copy_(q)
    rope = H.dev(rng.uniform(-1, 1, (3, 32, 2)).astype(np.float32))
    kv = H.dev(rng.normal(size=(3, 2, 64)), dt)
    for y in (q, wide):
        cache = torch.zeros((1, 2, 1, 18 * 64), dtype=torch.uint8, device="cuda")
        st = H.new_status()
        L.spec_rotary_append(y, kv, kv, H.dev(np.arange(3, dtype=np.int32)), H.dev(np.arange(3, dtype=np.int32)), rope,
                             y, cache, st)
        torch.cuda.synchronize()
        assert H.status(st) == 0
    assert torch.equal(q, wide)


def calls(torch, stream=None):
    L = H.lib()

    def i32(*s):
        return torch.zeros(s, dtype=torch.int32, device="cuda")

    def f32(*s):
        return torch.zeros(s, dtype=torch.float32, device="cuda")
    cache = torch.zeros((3, 2, 1, 18 * 64), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(L.spec_prefix_attention_workspace_bytes(4, 4, 2, 64), dtype=torch.uint8, device="cuda")
    x, q, st = f32(4, 2, 64), f32(4, 4, 64), i32(4)
    return [
        lambda: L.spec_rotary_append(q, x, x, i32(4), i32(4) - 1, f32(9, 32, 2), f32(4, 4, 64), cache, st, stream=stream),
        lambda: L.spec_prefix_attention(q, cache, i32(1, 2), i32(1) + 4, H.dev(np.array([0, 4], np.int32)), i32(1, 1),
                                        i32(1) + 7, H.dev(np.array([0, 1], np.int32)), f32(4, 4, 64), st, ws, 0.1,
                                        stream=stream),
        lambda: L.spec_sample(f32(1, 2, 8), f32(1, 2), i32(1, 2), st, stream=stream)]


def test_tensors_and_streams_of_another_device(torch, monkeypatch):
    L = H.lib()
    L._types()
    for call in calls(torch):
        call()
    for call in calls(torch, torch.cuda.Stream()):
        torch.cuda.synchronize()
        call()
    torch.cuda.synchronize()
    for call in calls(torch, types.SimpleNamespace(device_index=1, cuda_stream=0)):
        with pytest.raises(L.SpecError, match="stream"):
            call()
    these = calls(torch)
    monkeypatch.setattr(L, "_device", lambda: 1)
    for call in these:
        with pytest.raises(L.SpecError, match="cuda:1"):
            call()
