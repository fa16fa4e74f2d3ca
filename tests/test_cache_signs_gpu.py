"""The write into the 4-bit cache keeps the sign of a zero in every group, whichever way its
quotients are taken: the code of -0 is 8 wherever the group's scale is not 0 (spec_cache_append)."""
import numpy as np
import pytest

from test_cache_gpu import check, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_signs_of_zeros(torch, dtype):  # noqa: F811
    import serving as H
    rng = np.random.default_rng(1)
    x = H.rounded(rng.normal(size=(20, 2, 64)), dtype)
    zero = rng.random(x.shape)
    x[zero < 0.3] = -0.0
    x[zero > 0.8] = 0.0
    x[3, 0, :16] = -0.0                                  # a scale of 0: codes of 0
    x[4, 1, 16:32] *= 1e30                               # a scale at its largest
    x = H.rounded(x, dtype)
    slots = rng.permutation(32)[:20]
    st = check(torch, x, x[::-1].copy(), slots, np.zeros((2, 2, 1, 18 * 64), np.uint8), 0.01, 0.02, dtype)
    assert st == 0
