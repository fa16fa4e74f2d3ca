"""Sampling at the ends of its arguments' ranges: temperatures above 2^104, which count as that, and
min_p below the normal numbers.  Tokens, counts and log probabilities against float64, with the tolerances
of test_sample_gpu."""
import math

import numpy as np
import pytest

from oracle import serving as S
from tests import serving as H
from tests.test_sample_gpu import run, torch  # noqa: F401 (torch: a fixture)

pytestmark = pytest.mark.gpu
BIG = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("T", [1e30, 2e31, 1e32, 1e36, 1e37, 1e38, BIG])
def test_largest_temperatures(torch, T):  # noqa: F811
    """Logits of ordinary size are drawn from evenly; the largest ones still differ by more than any T."""
    rng = np.random.default_rng(1)
    T = float(np.float32(T))
    for x in (rng.normal(size=3000) * 5, rng.choice([-BIG, BIG, 0.5 * BIG, 0.0], 3000), rng.normal(size=3000) * 3e31):
        x = H.dev(x.astype(np.float32)[None, None])
        raw = x.double().cpu().numpy()[0, 0]
        for f in ({}, dict(top_k=70), dict(top_p=0.7), dict(min_p=0.3)):
            u = np.float32(rng.random())
            tokens, lp, kept, st = run(torch, x, [u], T, f.get("top_k"), f.get("top_p"), f.get("min_p"))
            g = {k: float(np.float32(v)) if isinstance(v, float) else v for k, v in f.items()}
            want, wl, wk, near = S.sample(raw, min(T, 2.0 ** 104), float(u), **g)
            assert near > 2.0 ** -32.9 or near == 0.0
            assert st == 0 and (tokens[0, 0], kept[0, 0]) == (want, wk), (T, f, tokens, want, kept, wk)
            assert abs(lp[0, 0] - wl) <= 2.0 ** -23 * abs(wl) + 2.0 ** -31


@pytest.mark.parametrize("min_p", [1e-37, 1.6e-38, 1e-38, 1e-39, 1e-41, 1e-44, 2e-45])
def test_smallest_min_p(torch, min_p):  # noqa: F811
    """Logits a few units in the last place around T ln(min_p)."""
    min_p = float(np.float32(min_p))
    for T in (1.0, 0.3, 7.0):
        T = float(np.float32(T))
        edge = np.float32(T * math.log(min_p))
        x = (edge + np.spacing(np.abs(edge)) * np.arange(-20, 21)).astype(np.float32)
        x = np.concatenate([[np.float32(0)], x])
        inside = np.longdouble(x) / np.longdouble(T) - np.log(np.longdouble(min_p))
        assert (np.abs(inside) > 1e-9).all()
        tokens, _, kept, st = run(torch, H.dev(x[None, None]), [0.5], T, None, None, min_p)
        assert st == 0 and tokens[0, 0] == 0 and kept[0, 0] == (inside >= 0).sum(), (T, kept, (inside >= 0).sum())
