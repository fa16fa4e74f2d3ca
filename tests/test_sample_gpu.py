"""Sampling (spec_sample) against the float64 oracle: tokens and counts are equal wherever no border
lies within 2^-32.9 of the mass, and no seed here has one: each weight is within 2^-34 of its value, so
a running sum and a part of the whole sum are each within 2^-34 of the mass, apart from half a unit
(2^-44 of the largest) an entry, which is less still in the flat rows where borders are dense.  Log probabilities: 2^-23 of their size (the rounding of a difference and of the result) and
2^-31 (weights, their sum and its logarithm within 2^-33 each)."""
import math

import numpy as np
import pytest

from oracle import serving as S
from tests import serving as H

pytestmark = pytest.mark.gpu
BAD_TEMP, BAD_LOGIT, BAD_FILTER = 4, 1024, 4096
FILTERS = [{}, dict(top_k=1), dict(top_k=7), dict(top_k=300), dict(top_k=10 ** 7), dict(top_p=0.0), dict(top_p=0.5),
           dict(top_p=0.95), dict(min_p=0.05), dict(min_p=1.0), dict(top_k=40, top_p=0.9),
           dict(top_k=1000, top_p=0.99, min_p=0.001), dict(top_p=0.9, min_p=0.2)]


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_draft_04_gb300 import build as B
    B.build()
    return t


def run(torch, x, u, T=None, k=None, p=None, m=None, stream=None):
    """x: logits on the GPU [B, n, V]; the settings per request."""
    B, n, _ = x.shape

    def vec(a, dtype):
        return None if a is None else H.dev(np.broadcast_to(np.asarray(a, dtype), (B,)))
    st = H.new_status()
    tokens, kept = (torch.full((B, n), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    lp = torch.full((B, n), 7.0, device="cuda")
    H.lib().spec_sample(x, H.dev(np.asarray(u, np.float32).reshape(B, n)), tokens, st, temperature=vec(T, np.float32),
                        top_k=vec(k, np.int32), top_p=vec(p, np.float32), min_p=vec(m, np.float32), logprob=lp,
                        kept=kept, stream=stream)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), lp.cpu().numpy(), kept.cpu().numpy(), H.status(st)


def check(torch, x, u, T=1.0, **f):
    """Every row of x [B, n, V] against the oracle, settings alike for all rows."""
    tokens, lp, kept, st = run(torch, x, u, T, f.get("top_k"), f.get("top_p"), f.get("min_p"))
    assert st == 0
    raw = x.double().cpu().numpy()
    u = np.asarray(u, np.float32).reshape(raw.shape[:2])
    for b, j in np.ndindex(*raw.shape[:2]):
        g = {k: float(np.float32(v)) if isinstance(v, float) else v for k, v in f.items()}
        want, wl, wk, near = S.sample(raw[b, j], float(np.float32(T)), float(u[b, j]), **g)
        assert near > 2.0 ** -32.9 or near == 0.0, "the seed has a border next to a decision"   # 0: equal weights, exact
        assert (tokens[b, j], kept[b, j]) == (want, wk), (b, j, f, tokens[b, j], want, kept[b, j], wk)
        assert abs(lp[b, j] - wl) <= 2.0 ** -23 * abs(wl) + 2.0 ** -31


def logits(torch, rng, shape, dtype, size=3.0):
    return H.dev(rng.normal(size=shape) * size, H.storage(torch, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 257, 1000, 2047, 2048, 2049, 4097, 20000])
def test_sizes_and_filters(torch, dtype, V):
    rng = np.random.default_rng(V)
    for i, f in enumerate(FILTERS):
        check(torch, logits(torch, rng, (3, 2, V), dtype), rng.random(6), T=(0.7, 1.0, 1.6)[i % 3], **f)


@pytest.mark.parametrize("dtype,V", [("bf16", 128256), ("f32", 151936), ("bf16", 700001), ("f32", 600000)])
def test_large_vocabularies(torch, dtype, V):
    """Slices that stay in shared memory, and (the last two) ones that do not."""
    rng = np.random.default_rng(V)
    x = logits(torch, rng, (2, 1, V), dtype, 2.0)
    for f in FILTERS[::2]:
        check(torch, x, rng.random(2), **f)


@pytest.mark.parametrize("rows", [1, 40, 160, 400])
def test_numbers_of_rows(torch, rows):
    """Clusters of one to eight CTAs a row."""
    rng = np.random.default_rng(rows)
    x = logits(torch, rng, (rows, 1, 9000), "bf16")
    for f in (FILTERS[0], FILTERS[7], FILTERS[10]):
        check(torch, x, rng.random(rows), T=0.8, **f)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 3, 5])
def test_rows_at_any_element(torch, dtype, pad):
    """Rows of views, whose first entries lie anywhere in 16 bytes."""
    rng = np.random.default_rng(pad)
    wide = logits(torch, rng, (3, 2, 5000 + pad), dtype)
    for f in (FILTERS[0], FILTERS[2], FILTERS[7]):
        check(torch, wide[..., :5000], rng.random(6), **f)
    check(torch, wide[:, 1:, :4999], rng.random(3), **FILTERS[11])


@pytest.mark.parametrize("V", [900, 6000, 40000])
@pytest.mark.parametrize("values", [1, 2, 5])
def test_ties(torch, V, values):
    """Thousands of equal entries next to every border: they go by their index."""
    rng = np.random.default_rng(V + values)
    x = H.dev(rng.integers(0, values, (2, 1, V)) * 0.5, torch.bfloat16)
    for f in FILTERS:
        check(torch, x, rng.random(2) * 0.999, T=0.9, **f)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_rows(torch, dtype):
    """-inf almost everywhere, the type's lowest value almost everywhere, and nothing but that."""
    rng = np.random.default_rng(3)
    lowest = float(torch.finfo(H.storage(torch, dtype)).min)
    for fill in (-math.inf, lowest):
        for few in (1, 5, 400):
            x = logits(torch, rng, (2, 1, 7000), dtype)
            off = np.ones((2, 1, 7000), bool)
            for b in range(2):
                off[b, 0, rng.permutation(7000)[:few]] = False
            x.masked_fill_(H.dev(off), fill)
            for f in FILTERS:
                check(torch, x, rng.random(2), **f)
    x = torch.full((1, 1, 3000), lowest, dtype=H.storage(torch, dtype), device="cuda")
    for f in FILTERS:
        check(torch, x, [0.4321], **f)
    x[..., 5:] = -math.inf
    for f in FILTERS:
        check(torch, x, [0.4321], **f)


@pytest.mark.parametrize("T", [1e-38, 1e-6, 0.03, 30.0, 1e6])
def test_temperatures(torch, T):
    rng = np.random.default_rng(8)
    x = logits(torch, rng, (2, 1, 5000), "f32")
    for f in FILTERS:
        check(torch, x, rng.random(2), T=T, **f)
    check(torch, x * 1e-3 + 40.0, rng.random(2), T=T, top_k=50)


def test_uniforms_at_the_ends(torch):
    rng = np.random.default_rng(9)
    x = logits(torch, rng, (1, 2, 3000), "f32")
    tokens, _, kept, st = run(torch, x, [0.0, np.float32(1) - np.float32(2.0 ** -24)], 1.0, k=20)
    order = np.argsort(-x[0].cpu().numpy(), axis=-1, kind="stable")[:, :20]
    assert st == 0 and tokens.tolist() == [[order[0].min(), order[1].max()]] and (kept == 20).all()


def test_settings_of_each_request(torch):
    """Requests' settings side by side, and rows that are not read."""
    rng = np.random.default_rng(10)
    B, V = 12, 6000
    x = logits(torch, rng, (B, 2, V), "bf16")
    k, p = rng.choice([0, -3, 1, 9, 200], B), rng.choice([1.0, 0.6, 0.9], B)
    m, T = rng.choice([0.0, 0.1], B), rng.choice([0.5, 1.0, 2.0], B)
    u = rng.random((B, 2)).astype(np.float32)
    u[::3, 1] = -1.0
    tokens, lp, kept, st = run(torch, x, u, T, k, p, m)
    assert st == 0
    raw = x.double().cpu().numpy()
    for b in range(B):
        for j in range(2):
            if u[b, j] == -1:
                assert tokens[b, j] == -1 and kept[b, j] == 0 and math.isnan(lp[b, j])
                continue
            want, wl, wk, near = S.sample(raw[b, j], T[b], float(u[b, j]), max(0, int(k[b])), float(np.float32(p[b])),
                                          float(np.float32(m[b])))
            assert near > 1e-9 and (tokens[b, j], kept[b, j]) == (want, wk)
            assert abs(lp[b, j] - wl) <= 2.0 ** -23 * abs(wl) + 2.0 ** -31


@pytest.mark.parametrize("what,bit", [("nan", BAD_LOGIT), ("inf", BAD_LOGIT), ("nothing", BAD_LOGIT), ("u", BAD_FILTER),
                                      ("u nan", BAD_FILTER), ("u one", BAD_FILTER), ("p", BAD_FILTER), ("p nan", BAD_FILTER),
                                      ("m", BAD_FILTER), ("T", BAD_TEMP), ("T nan", BAD_TEMP)])
@pytest.mark.parametrize("V", [300, 20000])
def test_bad_rows(torch, what, bit, V):
    rng = np.random.default_rng(11)
    x = logits(torch, rng, (3, 1, V), "f32")
    u, p, m, T = np.full(3, 0.3), np.full(3, 0.9), np.zeros(3), np.ones(3)
    nan = float("nan")
    if what == "nan":
        x[1, 0, V // 2] = nan
    if what == "inf":
        x[1, 0, V - 1] = math.inf
    if what == "nothing":
        x[1] = -math.inf
    for name, a, v in (("u", u, -0.5), ("u nan", u, nan), ("u one", u, 1.0), ("p", p, 1.1), ("p nan", p, nan),
                       ("m", m, -0.1), ("T", T, 0.0), ("T nan", T, nan)):
        if what == name:
            a[1] = v
    tokens, lp, kept, st = run(torch, x, u, T, [0, 0, 0], p, m)
    assert st == bit and tokens[1, 0] == -1 and kept[1, 0] == 0 and math.isnan(lp[1, 0])
    raw = x.double().cpu().numpy()
    for b in (0, 2):
        want, wl, wk, _ = S.sample(raw[b, 0], 1.0, float(np.float32(0.3)), top_p=float(np.float32(0.9)))
        assert (tokens[b, 0], kept[b, 0]) == (want, wk)


def test_captured_replayed_and_on_another_stream(torch):
    rng = np.random.default_rng(12)
    x = logits(torch, rng, (5, 1, 33000), "bf16")
    u, st = H.dev(rng.random((5, 1)).astype(np.float32)), H.new_status()
    p = H.dev(np.full(5, 0.9, np.float32))
    out = [torch.zeros((5, 1), dtype=torch.int32, device="cuda") for _ in range(3)]
    L = H.lib()
    L.spec_sample(x, u, out[0], st, top_p=p)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    L.spec_sample(x, u, out[1], st, top_p=p, stream=other)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.spec_sample(x, u, out[2], st, top_p=p)
    for _ in range(2):
        u.uniform_()
        g.replay()
        L.spec_sample(x, u, out[0], st, top_p=p)
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[2])
    assert H.status(st) == 0 and (out[1] >= 0).all()
