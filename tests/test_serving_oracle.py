"""Pins of the serving oracle (oracle/serving.py): each against a value worked by hand or a
route that does not share its formula."""
import math

import numpy as np
import pytest
from scipy.special import log_softmax, softmax

from oracle import serving as S


def test_levels_and_scales_are_the_4_and_8_bit_floats():
    assert len(S.SCALES) == 127 and S.SCALES[126] == 448.0 and S.SCALES[1] == 2.0 ** -9
    assert S.SCALES[0x38] == 1.0 and (np.diff(S.SCALES) > 0).all()
    # s e e m: exponent bias 1
    for c in range(1, 8):
        e, m = c >> 1, c & 1
        assert S.LEVELS[c] == (0.5 * m if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))


@pytest.mark.parametrize("x,code", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6),
                                    (5.0, 6), (0.26, 1), (0.24, 0), (5.01, 7), (4.99, 6), (9.0, 7)])
def test_ties_go_to_the_even_code(x, code):
    assert S.nearest_even(S.LEVELS, np.array([min(x, 6.0)]))[0] == code


def test_store_by_hand():
    # max 12, g = 0.5: scale 12 / 3 = 4; unit 2: 12 -> 6, -5 -> 2.5 -> 2, 3 -> 1.5, 0.4 -> 0.2 -> 0
    x = np.zeros(16)
    x[:4] = [12, -5, 3, 0.4]
    code, s = S.store(x, 0.5)
    assert S.SCALES[s] == 4.0
    assert list(code[:5]) == [7, 8 + 4, 3, 0, 0]
    assert list(S.values(code, s, 0.5)[:4]) == [12.0, -4.0, 3.0, 0.0]


def test_store_saturates_and_drops_what_is_below_the_scales():
    code, s = S.store(np.full(16, 1e9), 1.0)
    assert S.SCALES[s] == 448 and (code == 7).all()
    code, s = S.store(np.full(16, 1e-6), 1.0)
    assert s == 0 and (code == 0).all()
    code, s = S.store(np.array([np.nan] + [0.0] * 15), 1.0)
    assert s == 0 and (code == 0).all()


def test_store_error_is_within_half_a_level():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(2000, 16)).astype(np.float32)
    code, s = S.store(x, 0.01)
    r = S.SCALES[s] * np.float32(0.01)
    y = np.abs(x) / r[:, None]
    # gaps 0.5, 1, 2; beyond 6 the scale's rounding (1/16) clips at most 6 / 16
    half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0))
    assert (np.abs(np.abs(S.values(code, s, 0.01)) / r[:, None] - y) <= half + 1e-5).all()


def test_write_then_read_a_token():
    rng = np.random.default_rng(1)
    cache = np.zeros((3, 2, 2, 18 * 64), np.uint8)
    want = [S.write_token(cache, 2 * 32 + t, 1, w, rng.normal(size=64), 0.02)
            for t in range(20) for w in (0, 1)]
    for w in (0, 1):
        got = S.read_tokens(cache, np.array([2]), 1, 20, 64, w, 0.02)
        np.testing.assert_array_equal(got, np.array(want[w::2]))
    assert not cache[:2].any() and not cache[2, 0].any()


def test_pool_by_hand():
    # page 4; request 0 keeps 5 + 2 tokens (2 pages held), appends 3: 10 tokens, 3 pages;
    # request 1 is finished (2 pages back); request 2 shrinks from 3 pages to 2
    p = S.Pool(4, [9, 8], [[0, 1], [2, 3], [4, 5, 6]], 8)
    base, add, slots, pos = p.step([5, 6, 4], [1, 0, 0], [3, -1, 2], 100)
    assert base == [7, 0, 5] and add == [3, 0, 2]
    assert p.tables == [[0, 1, 9], [], [4, 5]] and p.free == [8, 2, 3, 6]
    assert pos == [7, 8, 9, 5, 6] and slots == [7, 36, 37, 21, 22]


def test_pool_refuses_in_order():
    p = S.Pool(4, [7], [[0], [1], [2]], 8)
    base, add, _, _ = p.step([4, 4, 2], None, [4, 1, 1], 100)
    assert add == [4, 0, 0]                       # the third would fit, but comes later
    p = S.Pool(4, [7, 8], [[0], [1]], 8)
    assert p.step([1, 1], None, [3, 2], 4)[1] == [3, 0]


def test_attention_against_scipy():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(3, 8)), rng.normal(size=(11, 8)), rng.normal(size=(11, 8))
    see = S.visible(3, 11)
    assert see.sum() == 9 + 10 + 11
    out, lse, _, _ = S.attention(q, k, v, see, 0.3)
    for i in range(3):
        x = 0.3 * q[i] @ k[see[i]].T
        np.testing.assert_allclose(out[i], softmax(x) @ v[see[i]], atol=1e-13)
        assert lse[i] == pytest.approx(math.log(math.fsum(np.exp(x))), abs=1e-13)


def test_tree_mask_and_empty_row():
    bits = np.array([[0b001], [0b011], [0]], np.uint32)
    see = S.visible(3, 3, bits)
    assert see.tolist() == [[True, False, False], [True, True, False], [False] * 3]
    out, lse, _, _ = S.attention(np.ones((3, 4)), np.ones((3, 4)), np.ones((3, 4)), see, 1.0)
    assert (out[2] == 0).all() and lse[2] == -math.inf and (out[0] == 1).all()


def test_logprobs_against_scipy():
    rng = np.random.default_rng(3)
    x = rng.normal(size=50) * 4
    x[7] = x[3]
    x[9] = -math.inf
    lp, H, ids, top, _ = S.logprobs(x, 0.7, 3, 50)
    want = log_softmax(x / 0.7)
    assert lp == pytest.approx(want[3], abs=1e-12)
    p = np.exp(want)
    assert H == pytest.approx(-np.sum(p[p > 0] * want[p > 0]), abs=1e-12)
    assert ids[-1] == 9 and list(ids).index(3) + 1 == list(ids).index(7)
    np.testing.assert_allclose(top, np.sort(want)[::-1], atol=1e-12)
    assert S.logprobs(np.full(4, -math.inf), 1.0, 0, 1) is None
    assert S.logprobs(np.array([1.0, math.inf]), 1.0, 0, 1) is None
