"""Log probabilities do not depend on a constant added to a row, whatever the constant and the
temperature (spec_logprobs).

Tolerance, derived before the first run (u = 2^-24), with no term in the size of the logits: an
entry's distance d from the maximum carries a few u |d|, its exponential 2^-22; sums of positive
numbers pass fewer than 64 roundings, 2^-18; ln Z one more of its own size.  So a log probability l
is off by 2^-18 + 2^-20 (1 + sum p |d|) + 2^-22 |l|, and the entropy by that and
2^-20 sum p d^2 + 2^-18 sum p |d|."""
import math

import numpy as np
import pytest

import serving as H
from oracle import serving as S
from test_logprobs_gpu import run, torch  # noqa: F401

pytestmark = pytest.mark.gpu
LOWEST = {"bf16": -3.3895313892515355e38, "f32": -3.4028234663852886e38}


def check(torch, x, tokens, T, K, dtype):  # noqa: F811
    """x: float64 values as stored, [B, n, V]; T: one number a request or None."""
    lp, ent, ids, top, st = run(torch, H.dev(x, H.storage(torch, dtype)), tokens, T, K)
    assert st == 0
    for b in range(x.shape[0]):
        t = 1.0 if T is None else float(np.float32(T[b]))
        for j in range(x.shape[1]):
            wl, we, wi, wt, m2 = S.logprobs(x[b, j], t, int(tokens[b, j]), K)
            d = (x[b, j] - x[b, j].max()) / t
            p = np.exp(d) / np.exp(d).sum()
            m1 = float(-(p * np.maximum(d, -1e4)).sum())
            tol = 2.0 ** -18 + 2.0 ** -20 * (1 + m1)

            def near(a, w):
                with np.errstate(over="ignore"):
                    w = float(np.float32(w))             # -inf below the 32-bit numbers
                return a == w or abs(a - w) <= tol + 2.0 ** -22 * abs(w)
            assert near(lp[b, j], wl), (b, j, lp[b, j], wl)
            assert abs(ent[b, j] - we) <= tol + 2.0 ** -20 * m2 + 2.0 ** -18 * m1, (b, j, ent[b, j], we)
            assert ids[b, j].astype(int).tolist() == wi.tolist()
            assert all(near(a, w) for a, w in zip(top[b, j], wt)), (b, j, top[b, j], wt)
    return lp, top


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [999, 5000, 40000])
def test_low_temperatures(torch, dtype, V):  # noqa: F811
    rng = np.random.default_rng(V)
    T = [1.0, 1e-1, 1e-2, 1e-3, 1e-4, 1e-5, 1e-6, 1e-8, 1e-20, 1e-30]
    x = 3 * rng.normal(size=(len(T), 2, V))
    x[..., 17] = 23.7                                    # the certain token of a nearly greedy row
    x[:, 1, 18] = 23.6
    x = H.rounded(x, dtype)
    tokens = np.full((len(T), 2), 17)
    lp, top = check(torch, x, tokens, T, 3, dtype)
    assert (lp <= 0).all() and (top <= 0).all()
    assert (np.abs(lp[2, 0]) <= 1e-6).all()              # (of the row beside it exp(-0.1 / 0.01) is left)
    assert (np.abs(lp[3:]) <= 1e-6).all() and (np.abs(top[3:, :, 0]) <= 1e-6).all()


def rows_of_one_value(torch, dtype, T, V):  # noqa: F811
    """As many equal entries as there are, at any level: -ln V each."""
    x = np.zeros((1, 8, V))
    for j, level in enumerate((0.0, 1e4, -1e4, -1e9, 1e9, -1e30, 1e30, LOWEST[dtype])):
        x[0, j] = level
    x = H.rounded(x, dtype)
    lp, _ = check(torch, x, np.arange(8).reshape(1, 8), [T], 3, dtype)
    assert np.abs(lp + math.log(V)).max() < 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0.6, 0.7, 1.0, 2.5])
@pytest.mark.parametrize("V", [999, 16384, 33333])
def test_rows_of_one_value(torch, dtype, T, V):  # noqa: F811
    rows_of_one_value(torch, dtype, T, V)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0.05, 0.7, 1.0])
def test_shifted_rows(torch, dtype, T):  # noqa: F811
    """Steps of 1/4 up to 16 and their sums with these constants are exact, as are bf16's steps of 8
    up to 256."""
    rng = np.random.default_rng(5)
    V = 20001
    if dtype == "bf16":
        base, shifts = 8.0 * rng.integers(-32, 1, V), (0, 1024, -1792)
    else:
        base, shifts = 0.25 * rng.integers(-64, 1, V), (0, 1000, -30000, 1e6)
    x = np.stack([base + s for s in shifts])[None]
    np.testing.assert_array_equal(x, H.rounded(x, dtype))
    tokens = np.full((1, len(shifts)), 4321)
    check(torch, x, tokens, [T], 5, dtype)
