"""Only a row's own entries count (spec_logprobs): not what fills the vectors beyond its ends, at
temperatures so high that every number is near every other one, and where all logits are as low as
a filler could be."""
import math

import numpy as np
import pytest

import serving as H
from test_logprobs_shift_gpu import check, rows_of_one_value, torch  # noqa: F401

pytestmark = pytest.mark.gpu
LOG2E = 1.4426950216293335                               # in 32 bits: its quotient is 1, products with that are exact


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 5, 999, 32000, 33000])
def test_high_temperatures(torch, dtype, V):  # noqa: F811
    rng = np.random.default_rng(V)
    T = [1e6, 1e20, 1e27, 1e28, 1e29, 1e30, 1e32, 1e35, 1e37]
    x = H.rounded(3 * rng.normal(size=(len(T), 2, V)), dtype)
    lp, _ = check(torch, x, np.zeros((len(T), 2), int), T, 1, dtype)
    assert np.abs(lp + math.log(V)).max() < 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [3, 999, 33000])
@pytest.mark.parametrize("T", [1.0, LOG2E, 1e28, 1e30])
def test_low_rows(torch, dtype, V, T):  # noqa: F811
    x = np.zeros((1, 4, V))
    for j, level in enumerate((-1e30, -1.0002e30, -2e30, -9e29)):
        x[0, j] = level
    lp, _ = check(torch, H.rounded(x, dtype), np.zeros((1, 4), int), [T], 1, dtype)
    assert np.abs(lp + math.log(V)).max() < 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [999, 16384, 33333])
def test_rows_of_one_value_without_roundings(torch, dtype, V):  # noqa: F811
    rows_of_one_value(torch, dtype, LOG2E, V)
