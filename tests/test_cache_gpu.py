"""The write into the 4-bit cache (spec_cache_append) against the format's definition
(oracle/serving.py): every byte of the cache and every value as stored are equal."""
import numpy as np
import pytest

import serving as H
from oracle import serving as S

pytestmark = pytest.mark.gpu
BAD_SLOT, BAD_KV = 512, 2048


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_draft_04_gb300 import build as B
    B.build()
    return t


def expect(cache, k, v, slots, gk, gv):
    """The cache after the call, and the values as stored (float64)."""
    cache = cache.copy()
    out = [np.zeros(k.shape), np.zeros(v.shape)]
    n = cache.shape[0] * cache.shape[2] * 16
    for t, slot in enumerate(slots):
        if 0 <= slot < n:
            for which, (x, g) in enumerate(((k, gk), (v, gv))):
                for h in range(k.shape[1]):
                    out[which][t, h] = S.write_token(cache, int(slot), h, which, x[t, h], g)
    return cache, out[0], out[1]


def run(torch, k, v, slots, cache, gk, gv, stored=True, stream=None):
    st = H.new_status()
    ks = torch.full(k.shape, 9.0, dtype=k.dtype, device="cuda") if stored else None
    vs = torch.full(v.shape, 9.0, dtype=v.dtype, device="cuda") if stored else None
    c = cache if hasattr(cache, "is_cuda") else H.dev(cache)
    H.lib().spec_cache_append(k, v, H.dev(slots.astype(np.int32)), c, st, gk, gv, k_stored=ks, v_stored=vs,
                              stream=stream)
    torch.cuda.synchronize()
    return c.cpu().numpy() if c.numel() < 1 << 30 else c, ks, vs, H.status(st)


def check(torch, k, v, slots, cache, gk, gv, dtype):
    dt = H.storage(torch, dtype)
    want, wk, wv = expect(cache, k, v, slots, gk, gv)
    got, ks, vs, st = run(torch, H.dev(k, dt), H.dev(v, dt), slots, cache, gk, gv)
    np.testing.assert_array_equal(got, want)
    # (code * scale) exact, times g rounded to fp32, rounded to the type
    for a, w in ((ks, wk), (vs, wv)):
        w32 = torch.from_numpy(w.astype(np.float32)).to(dt)
        assert torch.equal(a.cpu(), w32)
    return st


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H_,page", [(1, 1, 16), (7, 3, 32), (130, 2, 64), (33, 8, 128)])
def test_every_byte(torch, dtype, D, T, H_, page):
    rng = np.random.default_rng(T * D)
    pages = -(-T // page) + 2
    k = H.rounded(rng.normal(size=(T, H_, D)) * np.exp(rng.normal(size=(H_, D))), dtype)
    v = H.rounded(rng.normal(size=(T, H_, D)), dtype)
    slots = rng.permutation(pages * page)[:T]
    slots[rng.random(T) < 0.1] = -1
    cache = rng.integers(0, 256, (pages, H_, page // 16, 18 * D), dtype=np.uint8)   # left as it is elsewhere
    assert check(torch, k, v, slots, cache, 0.0137, 0.0021, dtype) == 0


@pytest.mark.parametrize("g", [1.0, 0.25, 1e-3, 2.0 ** -60, 2.0 ** 60, 0.37, 1.0 / 448])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes_of_numbers_and_scales(torch, g, dtype):
    """Groups from far below the smallest scale to far above the largest, ties on purpose."""
    rng = np.random.default_rng(3)
    T, D = 64, 64
    size = 10.0 ** rng.uniform(-6, 6, (T, 1, D // 16, 1)) * min(max(g, 1e-20), 1e20)
    x = rng.normal(size=(T, 1, D // 16, 16)) * size
    ties = rng.integers(-24, 25, (T, 1, D // 16, 16)) / 4.0 * min(max(g, 1e-20), 1e20)
    ties[..., 0] = 6.0 * min(max(g, 1e-20), 1e20)
    x = np.where(rng.random((T, 1, 1, 1)) < 0.5, x, ties).reshape(T, 1, D)
    k, v = H.rounded(x, dtype), H.rounded(x[::-1], dtype)
    cache = np.zeros((4, 1, 1, 18 * D), np.uint8)
    check(torch, k, v, rng.permutation(T), cache, float(np.float32(g)), float(np.float32(g)), dtype)


def test_extreme_numbers(torch):
    rng = np.random.default_rng(4)
    x = np.zeros((16, 1, 64), np.float32)
    x[0, 0, :16] = 3.0e38
    x[1, 0, :16] = 1e-45
    x[2, 0, 3] = -0.0
    x[3, 0, ::2] = -1e-30
    x[4, 0, 17] = 1e-38
    x[5, 0] = np.linspace(-3e38, 3e38, 64)
    for g in (1.0, 2.0 ** -60, 2.0 ** 60):
        assert check(torch, x, x, np.arange(16), np.zeros((1, 1, 1, 18 * 64), np.uint8), g, g, "f32") == 0


def test_not_finite(torch):
    x = np.ones((4, 1, 64), np.float32)
    x[0, 0, 3], x[1, 0, 20], x[2, 0, 40] = np.nan, np.inf, -np.inf
    want, wk, _ = expect(np.zeros((1, 1, 1, 18 * 64), np.uint8), x, x, np.arange(4), 0.5, 0.5)
    got, ks, _, st = run(torch, H.dev(x), H.dev(x), np.arange(4), np.zeros((1, 1, 1, 18 * 64), np.uint8), 0.5, 0.5)
    assert st == BAD_KV
    np.testing.assert_array_equal(got, want)
    assert ks[0, 0, 3] == 0 and ks[1, 0, 20] == 6 * 448 * 0.5 and ks[2, 0, 40] == -6 * 448 * 0.5
    np.testing.assert_array_equal(ks.cpu().numpy(), wk.astype(np.float32))


def test_slots_outside_the_cache(torch):
    rng = np.random.default_rng(5)
    x = H.rounded(rng.normal(size=(5, 2, 64)), "bf16")
    slots = np.array([0, 32, -2, 31, 2 ** 31 - 1])
    cache = np.zeros((2, 2, 1, 18 * 64), np.uint8)
    assert check(torch, x, x, slots, cache, 0.01, 0.01, "bf16") == BAD_SLOT


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides(torch, dtype):
    """Slices of a fused projection, and heads before tokens."""
    rng = np.random.default_rng(6)
    dt = H.storage(torch, dtype)
    T, Hk, D = 21, 2, 64
    k, v = H.rounded(rng.normal(size=(T, Hk, D)), dtype), H.rounded(rng.normal(size=(T, Hk, D)), dtype)
    slots = rng.permutation(48)[:T]
    cache = np.zeros((3, Hk, 1, 18 * D), np.uint8)
    want, _, _ = expect(cache, k, v, slots, 0.01, 0.02)
    qkv = torch.full((T, 5, D), float("nan"), dtype=dt, device="cuda")
    qkv[:, 1:3], qkv[:, 3:5] = H.dev(k, dt), H.dev(v, dt)
    got, _, _, st = run(torch, qkv[:, 1:3], qkv[:, 3:5], slots, cache, 0.01, 0.02, stored=False)
    np.testing.assert_array_equal(got, want)
    heads = H.dev(k.transpose(1, 0, 2), dt).transpose(0, 1)
    got, _, _, st2 = run(torch, heads, qkv[:, 3:5], slots, cache, 0.01, 0.02)
    np.testing.assert_array_equal(got, want)
    assert st == 0 and st2 == 0


def test_no_rows_and_many_rows(torch):
    rng = np.random.default_rng(7)
    cache = np.zeros((3, 1, 8, 18 * 64), np.uint8)
    x = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    got, _, _, st = run(torch, x, x, np.zeros(0), cache, 1.0, 1.0)
    assert st == 0 and not got.any()
    T = 5000                                             # more groups than one pass of the grid
    x = H.rounded(rng.normal(size=(T, 1, 64)), "bf16")
    cache = np.zeros((T // 128 + 1, 1, 8, 18 * 64), np.uint8)
    assert check(torch, x, x, rng.permutation(T), cache, 0.01, 0.01, "bf16") == 0


def test_offsets_beyond_2_to_the_32(torch):
    per = 4 * 8 * 18 * 128
    far = (5 << 30) // per
    cache = torch.zeros((far + 2, 4, 8, 18 * 128), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(8)
    k, v = (H.rounded(rng.normal(size=(6, 4, 128)), "bf16") for _ in range(2))
    slots = np.array([0, 15, 16, 127, 128, 200])
    want, _, _ = expect(np.zeros((2, 4, 8, 18 * 128), np.uint8), k, v, slots, 0.01, 0.02)
    dt = torch.bfloat16
    run(torch, H.dev(k, dt), H.dev(v, dt), slots + far * 128, cache, 0.01, 0.02)
    np.testing.assert_array_equal(cache[far:].cpu().numpy(), want)
    assert not cache[:4].any()


def test_another_stream(torch):
    rng = np.random.default_rng(9)
    x = H.rounded(rng.normal(size=(40, 2, 64)), "bf16")
    cache = np.zeros((4, 2, 1, 18 * 64), np.uint8)
    want, _, _ = expect(cache, x, x, np.arange(40), 0.01, 0.01)
    s = torch.cuda.Stream()
    got, _, _, _ = run(torch, H.dev(x, torch.bfloat16), H.dev(x, torch.bfloat16), np.arange(40), cache, 0.01, 0.01,
                       stream=s)
    np.testing.assert_array_equal(got, want)
