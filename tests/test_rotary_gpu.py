"""Norm, rotation and append in one pass (spec_rotary_append).  Queries: equal to the oracle's bit for
bit -- every step is one fp32 rounding, and the norm's factor is the rounded one unless the exact
value is within 2^-22 of a half ulp from its midpoint, which no seed here meets.  The cache and the
values as stored: equal to what spec_cache_append leaves for the oracle's keys."""
import numpy as np
import pytest

from oracle import serving as S
from tests import serving as H

pytestmark = pytest.mark.gpu
BAD_SLOT, BAD_KV, BAD_POSITION = 512, 2048, 8192
EPS = 1e-6


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_draft_04_gb300 import build as B
    B.build()
    return t


def table(rng, rows, R):
    a = rng.uniform(-1000, 1000, (rows, R // 2))
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def check(torch, qkv, Hq, Hkv, R, page=16, weights=True, interleaved=False, skip=(), eps=EPS, stored=True,
          in_place=False, status=0, seed=0):
    """qkv: [T, Hq + 2 Hkv, D] on the GPU, a fused projection's rows."""
    L, rng = H.lib(), np.random.default_rng(seed)
    T, _, D = qkv.shape
    dt = qkv.dtype
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    rope = table(rng, 50, R)
    positions = rng.integers(0, 50, T).astype(np.int32)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[list(skip)] = -1
    w = [H.dev(rng.normal(1, 0.3, D), dt) if weights else None for _ in range(2)]
    qh, kh = (x.float().cpu().numpy() for x in (q, k))
    want_q, want_k = (S.rotated(x, rope[positions], None if y is None else y.float().cpu().numpy(), eps, interleaved)
                      for x, y in zip((qh, kh), w))
    want_q, want_k = (torch.from_numpy(x).to(dt).cuda() for x in (want_q, want_k))
    caches = [torch.full((pages, Hkv, page // 16, 18 * D), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = (0.011, 0.003)
    kv = [[torch.full((T, Hkv, D), 7.0, dtype=dt, device="cuda") if stored else None for _ in range(2)] for _ in range(2)]
    st, st2 = H.new_status(), H.new_status()
    vv = v.clone()
    out = q if in_place else torch.full((T, Hq, D), 7.0, dtype=dt, device="cuda")
    L.spec_rotary_append(q, k, v, H.dev(positions), H.dev(slots), H.dev(rope), out, caches[0], st, *g, q_weight=w[0],
                         k_weight=w[1], eps=eps, interleaved=interleaved, k_stored=kv[0][0], v_stored=kv[0][1])
    L.spec_cache_append(want_k.contiguous(), vv, H.dev(slots), caches[1], st2, *g, k_stored=kv[1][0], v_stored=kv[1][1])
    torch.cuda.synchronize()
    assert H.status(st) == status and H.status(st2) == status
    left = torch.from_numpy(qh).to(dt).cuda() if in_place else torch.full_like(want_q, 7.0)
    want_q[list(skip)] = left[list(skip)]
    a, b = out.float(), want_q.float()
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
    assert torch.equal(caches[0], caches[1])
    if stored:
        assert torch.equal(kv[0][0], kv[1][0]) and torch.equal(kv[0][1], kv[1][1])


def rows(torch, T, heads, D, dtype, seed=0, size=1.0):
    rng = np.random.default_rng([T, heads, D, seed])
    return H.dev(rng.normal(size=(T, heads, D)) * size, H.storage(torch, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 96), (256, 256), (256, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_heads(torch, dtype, D, R, interleaved, weights):
    check(torch, rows(torch, 9, 8, D, dtype), 4, 2, R, interleaved=interleaved, weights=weights, page=32)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 1), (5, 5), (12, 4), (33, 3), (40, 8)])
@pytest.mark.parametrize("T", [1, 2, 17])
def test_head_counts(torch, Hq, Hkv, T):
    check(torch, rows(torch, T, Hq + 2 * Hkv, 128, "bf16"), Hq, Hkv, 128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tokens(torch, dtype):
    """Warps that go on to further heads of their token."""
    check(torch, rows(torch, 6000, 10, 64, dtype), 6, 2, 64, page=64, skip=(0, 5, 5999))


@pytest.mark.parametrize("in_place", [False, True])
def test_skipped_rows_and_place(torch, in_place):
    check(torch, rows(torch, 30, 8, 128, "bf16"), 4, 2, 128, skip=(0, 7, 29), in_place=in_place)
    check(torch, rows(torch, 30, 8, 128, "f32"), 4, 2, 64, skip=range(30), in_place=in_place)


def test_without_the_values_as_stored(torch):
    check(torch, rows(torch, 40, 8, 128, "bf16"), 4, 2, 128, stored=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e30])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
def test_sizes_of_numbers(torch, dtype, size, eps):
    """Squares that fp32 does not hold."""
    x = rows(torch, 6, 6, 64, dtype, size=size)
    x[2, :4] = 0
    x[3, :4, 5] = size * 1000
    if eps == 0:
        x[2, :4, 0] = size
    odd = BAD_KV if not torch.isfinite(x.float()).all() else 0
    check(torch, x, 2, 2, 64, eps=eps, status=odd)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_numbers_that_are_none(torch, dtype, value):
    x = rows(torch, 5, 6, 64, dtype)
    x[1, 0, 3] = value                                       # a query
    check(torch, x, 2, 2, 64)
    x[2, 2, 40] = value                                      # a key: with a norm its head, without one two elements
    x[3, 5, 1] = value                                       # a value
    check(torch, x, 2, 2, 64, status=BAD_KV)
    check(torch, x, 2, 2, 64, weights=False, status=BAD_KV)


def test_zero_heads_without_eps(torch):
    x = rows(torch, 3, 6, 64, "f32")
    x[1, :4] = 0                                             # 0 / 0
    check(torch, x, 2, 2, 64, eps=0.0, status=BAD_KV)


def test_bad_slots_and_positions(torch):
    L = H.lib()
    x = rows(torch, 6, 6, 64, "f32")
    args = dict(positions=np.array([0, 1, -1, 50, 2, 3], np.int32), slots=np.array([0, 64, 2, 3, -2, 5], np.int32))
    rope = table(np.random.default_rng(0), 50, 64)
    cache = torch.full((4, 2, 1, 18 * 64), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((6, 2, 64), 7.0, device="cuda")
    kv = [torch.full((6, 2, 64), 7.0, device="cuda") for _ in range(2)]
    st = H.new_status()
    L.spec_rotary_append(x[:, :2], x[:, 2:4], x[:, 4:], H.dev(args["positions"]), H.dev(args["slots"]), H.dev(rope), out,
                         cache, st, k_stored=kv[0], v_stored=kv[1])
    torch.cuda.synchronize()
    assert H.status(st) == BAD_SLOT | BAD_POSITION
    assert out[1:5].isnan().all() and torch.isfinite(out[[0, 5]]).all()
    assert all((t[1:5] == 0).all() and (t[[0, 5]] != 7).all() for t in kv)
    assert (cache[0, :, :, 64:96] == 0xA5).all() and (cache[1:] == 0xA5).all()      # tokens 2 and 3, other pages


def test_captured_and_on_another_stream(torch):
    L, rng = H.lib(), np.random.default_rng(0)
    x = rows(torch, 20, 8, 128, "bf16")
    pos, slots = H.dev(rng.integers(0, 50, 20).astype(np.int32)), H.dev(rng.permutation(32)[:20].astype(np.int32))
    rope, st = H.dev(table(rng, 50, 128)), H.new_status()
    outs = [(torch.zeros((20, 4, 128), dtype=x.dtype, device="cuda"),
             torch.zeros((2, 2, 1, 18 * 128), dtype=torch.uint8, device="cuda")) for _ in range(3)]

    def call(o, stream=None):
        L.spec_rotary_append(x[:, :4], x[:, 4:6], x[:, 6:], pos, slots, rope, o[0], o[1], st, stream=stream)
    call(outs[0])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    call(outs[1], other)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(outs[2])
    g.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])
