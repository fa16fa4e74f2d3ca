"""Borders of sampling among neighbouring values of the storage type, below 0 as above, where thousands of
entries share a value: more than a row's list holds, so the border is searched for in the row itself.
Against the float64 oracle, with the tolerances of test_sample_gpu."""
import numpy as np
import pytest

from tests import serving as H
from tests.test_sample_gpu import check, torch  # noqa: F401 (torch: a fixture)

pytestmark = pytest.mark.gpu
TOP_P = [dict(top_p=0.5), dict(top_p=0.8), dict(top_p=0.9), dict(top_p=0.95), dict(top_p=0.9, min_p=1e-4),
         dict(top_p=0.95, min_p=0.02)]


@pytest.mark.parametrize("mean,size", [(-10.0, 1.0), (-20.0, 2.0), (-9.0, 1.5), (10.0, 1.0)])
@pytest.mark.parametrize("V", [40000, 128256, 151936, 700001])
def test_flat_rows(torch, V, mean, size):  # noqa: F811
    """bf16 numbers between 8 and 16 are 1/16 apart.  700001: slices that do not stay in shared memory."""
    rng = np.random.default_rng([V, int(100 * abs(mean))])
    x = H.dev(rng.normal(mean, size, (1, 1, V)), torch.bfloat16)
    for f in TOP_P:
        check(torch, x, rng.random(1), **f)


@pytest.mark.parametrize("mean", [-10.0, 10.0])
def test_flat_rows_by_one_cta(torch, mean):  # noqa: F811
    """As many rows as give each one CTA; all of them are one row of memory, eight are looked at."""
    from oracle import serving as S
    from tests.test_sample_gpu import run
    rng = np.random.default_rng(17)
    V, rows = 128256, 640
    x = H.dev(rng.normal(mean, 1.0, (1, 1, V)), torch.bfloat16)
    u = rng.random(rows).astype(np.float32)
    tokens, _, kept, st = run(torch, x.expand(rows, 1, V), u, 1.0, None, 0.9, None)
    raw = x.double().cpu().numpy()[0, 0]
    assert st == 0
    for b in range(0, rows, 80):
        want, _, wk, near = S.sample(raw, 1.0, float(u[b]), 0, float(np.float32(0.9)), 0.0)
        assert near > 2.0 ** -32.9 and (tokens[b, 0], kept[b, 0]) == (want, wk)
    assert (kept == kept[0, 0]).all()


@pytest.mark.parametrize("V", [6000, 40000, 128256])
@pytest.mark.parametrize("values", [2, 5, 40])
@pytest.mark.parametrize("first", [-8.0, 8.0])
def test_ties_of_neighbouring_values(torch, V, values, first):  # noqa: F811
    """A few neighbouring bf16 values, each thousands of times."""
    rng = np.random.default_rng([V, values, int(first) + 100])
    sign = np.sign(first)
    x = H.dev(first + sign * rng.integers(0, values, (1, 1, V)) / 16.0, torch.bfloat16)
    for f in TOP_P + [{}, dict(top_k=20), dict(top_k=1500, top_p=0.7), dict(min_p=0.9)]:
        check(torch, x, rng.random(1) * 0.999, **f)


def test_flat_fp32_rows(torch):  # noqa: F811
    """The same in fp32, where wide ties are equal numbers."""
    rng = np.random.default_rng(18)
    x = H.dev(np.round(rng.normal(-10.0, 1.0, (1, 1, 100003)) * 16) / 16, torch.float32)
    for f in TOP_P:
        check(torch, x, rng.random(1), **f)
