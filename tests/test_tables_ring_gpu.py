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


@pytest.mark.parametrize("takes", [0, 5])
def test_a_ring_without_room_takes_nothing_back(torch, takes):  # noqa: F811
    """Pages that are said to be free and are held at once: entries of the ring that other requests
    take from are not written."""
    rng = np.random.default_rng(2)
    B = 300
    s = State(rng, B, 16, 200, 9, stride_slack=8)
    s.ring = rng.permutation(s.pages).astype(np.int32)
    s.tail = s.head + s.pages                            # all of them
    new = np.where(np.arange(B) % 3 == 0, -1, 0)
    new[1:1 + 3 * takes:3] = 40
    asked = np.maximum(0, -(-(s.seq + np.maximum(new, 0)) // s.page) - s.held)
    asked[new <= 0] = 0
    assert (asked.sum() > 0) == (takes > 0)
    got, st = call(torch, s, None, new, 40 * takes + 1)
    assert st == BAD_LEN
    np.testing.assert_array_equal(got["ring"], s.ring)
    np.testing.assert_array_equal(got["held"], s.held + asked)
    assert got["pos"].tolist() == [s.head + asked.sum(), s.tail] and got["ptr"][-1] == 40 * takes
    first = np.concatenate([[0], np.cumsum(asked)])
    for b in range(B):
        fresh = [s.ring[(s.head + i) % s.pages] for i in range(first[b], first[b + 1])]
        assert got["table"][b, :s.held[b] + asked[b]].tolist() == s.table[b, :s.held[b]].tolist() + fresh


def test_a_ring_that_fills_to_the_last_entry(torch):  # noqa: F811
    """Every page comes back: free and given pages are num_pages together."""
    rng = np.random.default_rng(3)
    s = State(rng, 50, 32, 300, 11)
    pool = s.pool()
    pool.step(s.seq, None, [-1] * 50, 1)
    got, st = call(torch, s, None, [-1] * 50, 1)
    head, tail = got["pos"]
    assert st == 0 and tail - head == s.pages
    assert [int(got["ring"][i % s.pages]) for i in range(head, tail)] == pool.free
