"""Rows of logits whose first and last vectors of 16 bytes are both partly filled, at every
alignment (spec_logprobs): the entries in them count like any other.  Widths at which one thread
holds both ends of a row are among them."""
import math

import numpy as np
import pytest

import serving as H
from test_logprobs_gpu import check, torch  # noqa: F401

pytestmark = pytest.mark.gpu
WIDTHS = [1023, 1025, 2047, 2049, 4095, 4097, 30725, 32769]


def rows(V, dtype):
    """Nine rows of an odd width, one after the other: every alignment of a row's first element."""
    rng = np.random.default_rng(V)
    x = 3 * rng.normal(size=(1, 9, V))
    x[..., :8] = 20 + 0.5 * np.arange(8)                 # the largest entries at both ends
    x[..., V - 1] = 30
    return H.rounded(x, dtype), rng.integers(0, V, (1, 9))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", WIDTHS)
def test_the_largest_entries_at_both_ends(torch, dtype, V):  # noqa: F811
    x, tokens = rows(V, dtype)
    tokens[0, ::2] = 0
    check(torch, x, tokens, [0.9], 12, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", WIDTHS)
def test_an_outlier_at_the_first_entry(torch, dtype, V):  # noqa: F811
    x, tokens = rows(V, dtype)
    x[..., 0] = 200
    check(torch, x, tokens, None, 3, dtype)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", WIDTHS)
def test_no_distribution_because_of_the_first_entry(torch, dtype, V, bad):  # noqa: F811
    x, tokens = rows(V, dtype)
    x[0, ::2, 0] = bad
    check(torch, x, tokens, None, 3, dtype)
