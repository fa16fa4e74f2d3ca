"""Sampling at temperatures near the resolution of the logits, where the distance at which a weight counts
as nothing is a few units in the last place of the largest logit.

The header's arithmetic in whole numbers: w = rint(2^43 exp((x - max) / T)), sums of them exact; the inputs
are such that no w 2^43 lies within 2^-30 of a half (the kernel's weights are within 2^-34 of theirs) but for
the entries of 0.  The uniform numbers keep a part of 2^-30 of the mass away from every border, or are 0, which
draws the first entry whose weight is not 0."""
import math

import numpy as np
import pytest

from tests import serving as H
from tests.test_sample_gpu import run, torch  # noqa: F401 (torch: a fixture)

pytestmark = pytest.mark.gpu
ONE = 2.0 ** 43


def oracle(x, T, u, top_p=1.0):
    """token, logprob, kept of float64 x."""
    d = (x - x.max()) / T
    w = np.exp(d) * ONE
    v = w[(w > 0.25) & (w < 2.0 ** 20)]                      # (one unit more or less of larger ones is 2^-20 of them)
    assert (np.abs(v - np.floor(v) - 0.5) > 2.0 ** -30 * np.maximum(1.0, v)).all()
    w = np.rint(w)
    order = np.lexsort((np.arange(len(x)), -x))
    total = w.sum()
    n = len(x)
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w[order])[:-1]])
        assert np.abs(before[1:] - top_p * total).min() > 2.0 ** -30 * total
        n = int((before < top_p * total).sum())
    kept = np.sort(order[:n])
    f = np.cumsum(w[kept])
    if u > 0:
        assert np.abs(f - u * f[-1]).min() > 2.0 ** -30 * f[-1]
    at = int((f <= u * f[-1]).sum())
    return int(kept[at]), d[kept[at]] - math.log(f[-1] / ONE), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [20.0, 16.0, 2.0 ** -20 - 16.0, 300.0, -300.0, 1e4, 1e6, 1.5])
def test_few_units_in_the_last_place(torch, m, dtype):  # noqa: F811
    rng = np.random.default_rng(int(abs(m)) + 1)
    V = 3000
    ulp = float(np.spacing(np.float32(abs(m))))
    for part in np.geomspace(0.4, 40.0, 24):
        T = np.float32(part * ulp / 31.5)
        x = np.full(V, m) - ulp * rng.integers(1, 60, V)
        x[rng.permutation(V)[:7]] = m
        x[:V // 2].sort()                                    # u = 0 draws the smallest number whose weight is not 0
        x = H.dev(x.astype(np.float32)[None, None], H.storage(torch, dtype))
        raw = x.double().cpu().numpy()[0, 0]
        for u in (0.0, 0.37, 0.99):
            u = float(np.float32(u))
            for p in (1.0, float(np.float32(0.7))):
                tokens, lp, kept, st = run(torch, x, [u], T, None, p)
                want, wl, wk = oracle(raw, float(T), u, p)
                assert st == 0 and (tokens[0, 0], kept[0, 0]) == (want, wk), (part, u, p, tokens, want, kept, wk)
                assert abs(lp[0, 0] - wl) <= 2.0 ** -23 * abs(wl) + 2.0 ** -31


@pytest.mark.parametrize("V", [20000, 151936])
def test_many_entries_of_no_weight(torch, V):  # noqa: F811
    """All entries but one far below the largest in units of T: none is ever drawn."""
    for m, parts in ((20.0, (0.6, 1.2, 1.49, 2.4)), (1e4, (0.6, 1.2, 1.49, 2.4)), (16.0, (0.3, 0.6, 0.74, 1.4))):
        ulp = float(np.spacing(np.float32(m)))
        for part in parts:
            T = np.float32(part * ulp / 31.5)
            x = torch.full((1, 4, V), m - 3 * ulp, device="cuda")
            x[..., V - 5] = m
            for p in (1.0, 0.9):
                tokens, lp, kept, st = run(torch, x, [0.0, 1e-6, 0.5, 1 - 2.0 ** -24], T, None, p)
                assert st == 0 and (tokens == V - 5).all() and (kept == (V if p == 1.0 else 1)).all()
                assert (np.abs(lp) <= 2.0 ** -31).all()
