"""Temperatures below the normal 32-bit numbers are finite and above 0, so a row has a distribution
(spec_logprobs)."""
import numpy as np
import pytest

import serving as H
from test_logprobs_shift_gpu import check, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [7, 999, 33000])
def test_subnormal_temperatures(torch, dtype, V):  # noqa: F811
    rng = np.random.default_rng(V)
    T = [1.2e-38, 4.3e-39, 4.2e-39, 1e-39, 1e-42, 2e-45]
    x = 3 * rng.normal(size=(len(T), 3, V))
    x[..., 3] = 23.7
    x[:, 1] = -1 - np.abs(x[:, 1])                       # all below 0
    x[:, 1, 2] = -0.5
    x[:, 2] = 1e-39 * rng.integers(-9, 9, V)             # logits of the temperatures' size
    x[:, 2, V - 1] = 2e-38
    x = H.rounded(x, dtype)
    tokens = np.tile(x[0].argmax(-1), (len(T), 1))
    lp, _ = check(torch, x, tokens, T, 2, dtype)
    assert (lp[:, :2] <= 0).all() and (lp[:, 0] >= -1e-6).all()
