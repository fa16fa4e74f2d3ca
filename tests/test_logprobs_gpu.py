"""Log probabilities, entropy and top alternatives (spec_logprobs) against the float64 oracle.

Tolerances, derived before the first run (u = 2^-24): x = logit / T carries up to 2 u |x|; an
exponential carries 2^-22 and its argument's 4 u |d|; so lse is off by at most
2^-21 (2 + |lse| + max|x| + sum p |d|), with sum p |d| <= 1 + sum p d^2 / 1, and the log
probabilities by that and their own difference.  The entropy's second term sums p d, each off by
p |d| (2^-22 + 4 u |d|): 2^-20 (1 + H + sum p d^2).  The ids are equal."""
import math

import numpy as np
import pytest

import serving as H
from oracle import serving as S

pytestmark = pytest.mark.gpu
BAD_TOKEN, BAD_TEMP, BAD_LOGIT = 1, 4, 1024


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_draft_04_gb300 import build as B
    B.build()
    return t


def run(torch, logits, tokens, T, K, stream=None):
    L = H.lib()
    B, n, V = logits.shape
    st = H.new_status()

    def f(*s, dt=torch.float32):
        return torch.full(s, -55, dtype=dt, device="cuda")
    lp, ent = f(B, n), f(B, n)
    ids, top = (f(B, n, K, dt=torch.int32), f(B, n, K)) if K else (None, None)
    ws = torch.full((L.spec_logprobs_workspace_bytes(B * n, V, K),), 0x5A, dtype=torch.uint8, device="cuda")
    L.spec_logprobs(logits, H.dev(np.asarray(tokens, np.int32).reshape(B, n)), lp, ent, st, ws,
                    temperature=None if T is None else H.dev(np.asarray(T, np.float32)), top_ids=ids,
                    top_logprobs=top, stream=stream)
    torch.cuda.synchronize()
    c = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    return c(lp), c(ent), c(ids), c(top), H.status(st)


def check(torch, x, tokens, T, K, dtype, logits=None, **kw):
    """x: float64 values as stored, [B, n, V]."""
    B, n, V = x.shape
    tokens = np.asarray(tokens).reshape(B, n)
    logits = H.dev(x, H.storage(torch, dtype)) if logits is None else logits
    lp, ent, ids, top, st = run(torch, logits, tokens, T, K, **kw)
    bits = 0
    for b in range(B):
        t = 1.0 if T is None else float(np.float32(T[b]))
        for j in range(n):
            tok = int(tokens[b, j])
            want = None if tok < 0 or tok >= V else S.logprobs(x[b, j], t, tok, K)
            if want is None:
                bits |= 0 if tok == -1 else BAD_TOKEN if tok < 0 or tok >= V else BAD_LOGIT
                assert np.isnan(lp[b, j]) and np.isnan(ent[b, j])
                assert K == 0 or ((ids[b, j] == -1).all() and np.isnan(top[b, j]).all())
                continue
            wl, we, wi, wt, m2 = want
            fin = np.isfinite(x[b, j])
            xs = np.abs(x[b, j][fin] / t).max()
            tol = 2.0 ** -21 * (3 + 2 * xs + m2)

            def near(a, w):
                return a == w or abs(a - w) <= tol + 2.0 ** -22 * abs(w)
            assert near(lp[b, j], wl), (lp[b, j], wl, tol)
            assert abs(ent[b, j] - we) <= 2.0 ** -20 * (1 + we + m2) + tol, (ent[b, j], we)
            if K:
                assert ids[b, j].astype(int).tolist() == wi.tolist()
                assert all(near(a, w) for a, w in zip(top[b, j], wt))
    assert st == bits
    return lp, ent, ids, top


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 16, 31, 100, 1000, 4095, 4097, 16384, 16385, 32000, 50257])
def test_vocabularies(torch, dtype, V):
    rng = np.random.default_rng(V)
    x = H.rounded(3 * rng.normal(size=(2, 3, V)), dtype)
    tokens = rng.integers(0, V, (2, 3))
    tokens[1, 2] = -1
    check(torch, x, tokens, [0.7, 1.3], min(V, 20), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [128256, 151936, 300001])
def test_large_vocabularies(torch, dtype, V):
    rng = np.random.default_rng(V)
    x = H.rounded(3 * rng.normal(size=(1, 3, V)), dtype)
    check(torch, x, [[5, V - 1, 77]], None, 32, dtype)


@pytest.mark.parametrize("K", [0, 1, 2, 5, 8, 20, 31, 32])
def test_numbers_of_alternatives(torch, K):
    rng = np.random.default_rng(K)
    x = H.rounded(2 * rng.normal(size=(3, 2, 5000)), "bf16")
    check(torch, x, rng.integers(0, 5000, (3, 2)), [0.5, 1.0, 2.0], K, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 3000, 40000])
def test_ties_go_to_the_lower_index(torch, dtype, V):
    rng = np.random.default_rng(V)
    x = np.zeros((1, 6, V))
    x[0, 1] = rng.integers(0, 3, V)                      # many equal maxima
    x[0, 2, V // 2:] = 1.0
    x[0, 3] = np.arange(V) // 7
    x[0, 4] = -(np.arange(V) // 3)
    x[0, 5] = np.where(rng.random(V) < 0.5, 0.0, -0.0)   # zeros of either sign are equal
    x = H.rounded(x, dtype)
    check(torch, x, [[0, 1, 2, 3, 4, 5]], None, 32, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [70000, 2000])
def test_orders_that_crowd_the_alternatives(torch, dtype, V):
    """Ascending, descending, and the largest entries at one stride or in one run."""
    rng = np.random.default_rng(V)
    x = np.zeros((1, 7, V))
    x[0, 0], x[0, 1] = np.linspace(-20, 20, V), np.linspace(20, -20, V)
    for j, s in enumerate((64, 256, 2048)):
        x[0, 2 + j] = rng.normal(size=V)
        x[0, 2 + j, 5::s] += 20
    x[0, 5] = rng.normal(size=V)
    x[0, 5, 300:700] += 15
    x[0, 6] = rng.normal(size=V)
    x[0, 6, 8 * 17::8] += 9
    check(torch, H.rounded(x, dtype), rng.integers(0, V, (1, 7)), None, 32, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_and_extreme_logits(torch, dtype):
    rng = np.random.default_rng(1)
    V = 9000
    x = 3 * rng.normal(size=(2, 6, V))
    x[0, 0, rng.random(V) < 0.9] = -math.inf             # a grammar's mask
    x[0, 1] = -math.inf
    x[0, 1, 4321] = 2.0                                  # one choice
    x[0, 2, ::2] = -3.3e38                               # the type's lowest values as a mask
    x[0, 3] = -3.3e38
    x[0, 3, 7] = 0.0
    x[0, 4] = 1e4 * rng.normal(size=V)
    x[0, 5] += 3e38 / 1.1
    x[1, 0] = 1e-30 * rng.normal(size=V)
    x[1, 1, 0] = -math.inf
    x[1, 2, V - 1] = -math.inf
    x[1, 3] = np.where(np.arange(V) < 3, x[1, 3], -math.inf)
    x = H.rounded(x, dtype)
    check(torch, x, [[5, 4321, 7, 8, 9, 10], [1, 0, V - 1, 2, 3, 4]], None, 8, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 5, 8000, 33332])
def test_rows_without_a_distribution(torch, dtype, at):
    rng = np.random.default_rng(2)
    V = 33333
    x = H.rounded(rng.normal(size=(1, 5, V)), dtype)
    x[0, 0, at], x[0, 1, at], x[0, 2] = math.nan, math.inf, -math.inf
    x[0, 4, at] = -math.nan
    check(torch, x, [[1, 2, 3, 4, at]], None, 5, dtype)


def test_bad_tokens_and_temperatures(torch):
    rng = np.random.default_rng(3)
    x = H.rounded(rng.normal(size=(4, 3, 100)), "bf16")
    check(torch, x[:1], [[100, -2, 99]], None, 3, "bf16")
    lp, ent, ids, top, st = run(torch, H.dev(x, torch.bfloat16), np.full((4, 3), 5),
                                [0.0, -1.0, math.nan, math.inf], 3)
    assert st == BAD_TEMP and np.isnan(lp).all() and np.isnan(ent).all() and (ids == -1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [999, 20001])
def test_strides_and_alignment(torch, dtype, V):
    """Rows that start anywhere: odd widths, columns of a wider buffer, a step between requests."""
    rng = np.random.default_rng(V)
    dt = H.storage(torch, dtype)
    x = H.rounded(rng.normal(size=(3, 2, V)), dtype)
    tokens = rng.integers(0, V, (3, 2))
    for lead, pad in ((0, 1), (8, 3), (16, 0)):
        wide = torch.full((3, 4, lead + V + pad), float("nan"), dtype=dt, device="cuda")
        wide[:, 1:3, lead:lead + V] = H.dev(x, dt)
        view = wide[:, 1:3, lead:lead + V]
        if view.data_ptr() % 16:
            continue
        check(torch, x, tokens, None, 7, dtype, logits=view)
    flip = H.dev(x.transpose(1, 0, 2), dt).transpose(0, 1)
    check(torch, x, tokens, None, 7, dtype, logits=flip)


def test_rows_that_are_not_read(torch):
    """Padding rows may hold anything."""
    x = np.full((2, 2, 5000), math.nan)
    x[0, 0] = np.linspace(0, 1, 5000)
    check(torch, H.rounded(x, "f32"), [[3, -1], [-1, -1]], [1.0, 1.0], 4, "f32")


def test_many_rows_and_another_stream(torch):
    rng = np.random.default_rng(4)
    x = H.rounded(rng.normal(size=(900, 2, 37)), "f32")
    tokens = rng.integers(-1, 37, (900, 2))
    a = check(torch, x, tokens, rng.uniform(0.5, 2, 900), 3, "f32")
    b = check(torch, x, tokens, None, 0, "f32", stream=torch.cuda.Stream())
    assert a[2] is not None and b[2] is None


def test_offsets_beyond_2_to_the_32(torch):
    rows, V = 34000, 128256                              # 8.7 GB of bf16
    L = H.lib()
    x = torch.zeros((rows, 1, V), dtype=torch.bfloat16, device="cuda")
    x[-1, 0, 777] = 5.0
    x[-1, 0, V - 1] = 3.0
    tokens = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    tokens[-1] = V - 1
    lp, ent = (torch.zeros((rows, 1), device="cuda") for _ in range(2))
    ids, top = torch.zeros((rows, 1, 3), dtype=torch.int32, device="cuda"), torch.zeros((rows, 1, 3), device="cuda")
    ws = torch.empty(L.spec_logprobs_workspace_bytes(rows, V, 3), dtype=torch.uint8, device="cuda")
    L.spec_logprobs(x, tokens, lp, ent, H.new_status(), ws, top_ids=ids, top_logprobs=top)
    row = np.zeros(V)
    row[777], row[V - 1] = 5.0, 3.0
    want = S.logprobs(row, 1.0, V - 1, 3)
    assert ids[-1, 0].tolist() == [777, V - 1, 0]
    assert abs(lp[-1, 0].item() - want[0]) < 1e-5 and abs(ent[-1, 0].item() - want[1]) < 1e-5
    assert torch.isnan(lp[:-1]).all()
