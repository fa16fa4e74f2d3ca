"""The serving calls launch on the current device: tensors and streams of another one are refused
before anything is enqueued.  One GPU stands for two: the binding is told that another one is
current."""
import types

import numpy as np
import pytest

import serving as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def calls(torch, stream=None):
    L = H.lib()

    def i32(*s):
        return torch.zeros(s, dtype=torch.int32, device="cuda")

    def f32(*s):
        return torch.zeros(s, dtype=torch.float32, device="cuda")
    cache = torch.zeros((3, 2, 1, 18 * 64), dtype=torch.uint8, device="cuda")
    ring = torch.zeros(2, dtype=torch.int64, device="cuda")
    ws = torch.zeros(max(L.spec_cache_attention_workspace_bytes(4, 2, 64), 1 << 16), dtype=torch.uint8, device="cuda")
    x, st = f32(4, 2, 64), i32(4)
    return [
        lambda: L.spec_block_tables(i32(2), None, i32(2), i32(2), ring, i32(3), i32(2, 2), i32(2), i32(2), i32(2),
                                    ring.clone(), i32(3), i32(4), i32(4), st, 16, stream=stream),
        lambda: L.spec_cache_append(x, x, i32(4), cache, st, stream=stream),
        lambda: L.spec_cache_attention(f32(4, 4, 64), cache, i32(1, 2), i32(1) + 4, H.dev(np.array([0, 4], np.int32)),
                                       f32(4, 4, 64), st, ws, 0.1, stream=stream),
        lambda: L.spec_logprobs(f32(1, 2, 8), i32(1, 2), f32(1, 2), f32(1, 2), st, ws, stream=stream)]


def test_the_calls_run(torch):
    for call in calls(torch):
        call()
    for call in calls(torch, torch.cuda.Stream()):
        torch.cuda.synchronize()
        call()
    torch.cuda.synchronize()


def test_tensors_of_another_device(torch, monkeypatch):
    L = H.lib()
    L._types()
    these = calls(torch)
    monkeypatch.setattr(L, "_device", lambda: 1)
    for call in these:
        with pytest.raises(L.SpecError, match="cuda:1"):
            call()


def test_a_workspace_of_another_device(torch):
    L = H.lib()
    L._types()
    t = torch.zeros(64, dtype=torch.uint8, device="cuda")
    assert L._args.addresses(0, "workspace", t, None, None) == (t.data_ptr(), 64)
    with pytest.raises(L.SpecError, match="workspace is on cuda:0"):
        L._args.addresses(1, "workspace", t, None, None)


def test_a_stream_of_another_device(torch):
    L = H.lib()
    for call in calls(torch, types.SimpleNamespace(device_index=1, cuda_stream=0)):
        with pytest.raises(L.SpecError, match="stream"):
            call()
