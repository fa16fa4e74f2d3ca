"""Shared prefixes with more rows a request: blocks whose tables have room for long contexts (16- and 32-row
tiles for the requests' own tokens), and whole prompts behind a prefix.  Oracle and tolerances as in
test_prefix_attention_gpu."""
import numpy as np
import pytest

from tests.test_prefix_attention_gpu import Shared, check, torch  # noqa: F401 (torch: a fixture)

pytestmark = pytest.mark.gpu


def with_room(table, page, tokens):
    """The same tables, wide enough for `tokens`."""
    wide = np.full((len(table), tokens // page + 1), -1, np.int32)
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 6, 7, 8, 9, 20])
@pytest.mark.parametrize("room", [4096, 32768])
def test_blocks_in_large_tables(torch, D, n, room):  # noqa: F811
    """4 n rows a request and key-value head: every tile of the plain call."""
    rng = np.random.default_rng([D, n])
    lens = n + rng.integers(0, 150, 6)
    s = Shared(rng, [4, 2], [200, 45], lens, [n] * 6, 8, 2, D, 32, "bf16")
    check(torch, s, table=with_room(s.p.table[:6], 32, room))


@pytest.mark.parametrize("n", [5, 7])
def test_long_own_contexts(torch, n):  # noqa: F811
    """Own tokens that are shared out among warps, and joined."""
    rng = np.random.default_rng(n)
    check(torch, Shared(rng, [2, 1], [1000, 300], [5000, 33, 2600], [n] * 3, 8, 2, 128, 64, "bf16"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,page", [(64, 128), (128, 32), (256, 64)])
def test_prompts_behind_prefixes(torch, dtype, D, page):  # noqa: F811
    """Requests' own prompts, the first step after a prefix, beside ones that go on with a few tokens."""
    rng = np.random.default_rng(D)
    news = np.array([100, 517, 1, 260, 33, 129])
    context = np.array([0, 0, 70, 0, 5, 300])
    check(torch, Shared(rng, [3, 1, 2], [300, 0, 1111], news + context, news, 4, 2, D, page, dtype))


def test_one_long_prompt(torch):  # noqa: F811
    rng = np.random.default_rng(3)
    check(torch, Shared(rng, [1], [2050], [2000], [2000], 4, 1, 128, 64, "bf16"))
