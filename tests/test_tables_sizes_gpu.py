"""Every number of requests finds its shared memory (spec_block_tables): also those whose prefix sums
nearly fill what a launch gets without asking."""
import numpy as np
import pytest

from test_tables_gpu import State, call, check, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [1637, 1638, 2400, 2429, 2430, 2431, 2432, 2444, 2456, 2457, 2458, 4095])
def test_numbers_of_requests(torch, B):  # noqa: F811
    rng = np.random.default_rng(B)
    s = State(rng, B, 16, 40, B)
    accept, new = rng.integers(-1, 8, B), rng.integers(-1, 9, B)
    rows = int(np.maximum(new, 0).sum())
    pool = s.pool()
    want = pool.step(s.seq, accept, new, rows)
    got, st = call(torch, s, accept, new, rows)
    assert st == 0
    check(s, got, *want, pool, rows)
