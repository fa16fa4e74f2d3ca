"""A ring of free pages that cannot be (spec_block_tables): nothing is written into it, and requests
keep the pages that they would have given back."""
import numpy as np
import pytest

from test_tables_gpu import BAD_LEN, State, call, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("head,tail", [(0, -1), (-1, 3), (7, 6), (2 ** 40, 2 ** 40 + 10 ** 6), (5, -2 ** 62)])
def test_a_refused_ring_is_not_written(torch, head, tail):  # noqa: F811
    rng = np.random.default_rng(1)
    s = State(rng, 30, 16, 200, 9)
    s.ring = rng.permutation(s.pages).astype(np.int32)
    s.head, s.tail = head, tail
    new = np.where(np.arange(30) % 3 == 0, -1, 0)        # finished ones, and ones that shrink
    got, st = call(torch, s, None, new, 8)
    assert st == BAD_LEN
    np.testing.assert_array_equal(got["ring"], s.ring)
    np.testing.assert_array_equal(got["table"], s.table)
    np.testing.assert_array_equal(got["held"], s.held)
    np.testing.assert_array_equal(got["kv"], np.where(new < 0, 0, s.seq))
    assert got["pos"].tolist() == [head, tail] and got["ptr"][-1] == 0
