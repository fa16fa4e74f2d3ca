"""Attention over the 4-bit paged cache (spec_cache_attention) against the float64 oracle
(oracle/serving.py), which reads the same bytes.

Tolerances, derived before the first run (u = 2^-24):
* a score is a dot product of D exact products added in fp32, at most D / 16 + 4 <= 20 roundings or
  truncations (2 u) of partial sums bounded by A = scale sum |q||k|, and two roundings of its scale:
  its error is below 42 u A < 2^-18 A; fp32 queries in two 11-bit terms lose 2^-22 of |q|, inside that.
* a probability's relative error is at most twice that plus its rounding: 2^-11 to 11 bits (bf16
  queries; 2^-12 to nearest, and the sum's own share), 2^-20 in two terms (fp32); the weighted sums
  add up to 2^-15 of sum p |v| over the longest case's tokens (additions per 16 tokens, in fp32).
* the output rounds once: 2^-8 |out| covers half a bf16 ulp, 2^-22 fp32's.
* lse: the score's error, and 2^-20 (1 + |lse|) for the exponentials, the sum and the logarithm."""
import numpy as np
import pytest

import serving as H
from oracle import serving as S

pytestmark = pytest.mark.gpu
BAD_LEN, BAD_SLOT = 2, 512


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_draft_04_gb300 import build as B
    B.build()
    return t


def check(torch, p, scale=None, floor=0.0, **kw):
    scale = 1.0 / np.sqrt(p.D) if scale is None else scale
    out, lse, st = p.run(torch, scale, **kw)
    want, wlse, tol_o, tol_l = p.oracle(scale)
    assert st == 0
    bad = ~(np.abs(out - want) <= tol_o + floor)
    assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5], want[bad][:5], tol_o[bad][:5])
    if lse is not None:
        inf = np.isneginf(wlse)
        assert np.array_equal(np.isneginf(lse), inf)
        off = np.abs(lse[~inf] - wlse[~inf])
        assert (off <= tol_l[~inf]).all(), off.max()
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_types_heads_pages(torch, dtype, D, page):
    rng = np.random.default_rng(D + page)
    p = H.Paged(rng, [1, 17, 64, 130, 333], [1, 1, 3, 2, 8], 6, 2, D, page, dtype)
    check(torch, p)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257, 1000])
def test_single_token_lengths(torch, L):
    rng = np.random.default_rng(L)
    check(torch, H.Paged(rng, [L], [1], 4, 2, 64, 32, "bf16"))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (8, 1), (5, 5), (12, 4), (16, 1), (24, 1), (40, 1)])
@pytest.mark.parametrize("n", [1, 7, 16])
def test_head_groups(torch, Hq, Hkv, n):
    rng = np.random.default_rng(Hq * 100 + n)
    check(torch, H.Paged(rng, [40 + n, n, 90], [n, n, n], Hq, Hkv, 64, 16, "bf16"))


@pytest.mark.parametrize("n", [2, 33, 65, 150, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_blocks_of_many_rows(torch, n, dtype):
    """Row tiles beyond one, with the causal edge inside each of them."""
    rng = np.random.default_rng(n)
    check(torch, H.Paged(rng, [n, n + 37], [n, n], 4, 2, 128, 64, dtype))


@pytest.mark.parametrize("n", [5, 25, 64, 70, 129])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_masks(torch, n, dtype):
    rng = np.random.default_rng(n)
    check(torch, H.Paged(rng, [n, n + 1, n + 50, n + 200], [n] * 4, 4, 1, 64, 32, dtype, tree=H.tree_of()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(torch, dtype):
    """No context and no bit in the row's mask: zeros and -inf."""
    rng = np.random.default_rng(5)
    p = H.Paged(rng, [9, 40, 25], [9, 9, 25], 4, 2, 64, 16, dtype, tree=H.tree_of(empty=True))
    out, lse = check(torch, p)
    assert (out[4] == 0).all() and np.isneginf(lse[4]).all()
    assert np.isfinite(lse[9 + 4]).all()                 # context is still seen


def test_mask_bits_beyond_the_rows_are_ignored(torch):
    rng = np.random.default_rng(6)
    p = H.Paged(rng, [30, 31], [5, 6], 2, 1, 64, 16, "bf16", tree=H.tree_of())
    a, _, _ = p.run(torch, 0.125)
    p.mask = np.concatenate([p.mask | np.uint32(0xFFFFFF80), np.full_like(p.mask, 0xFFFFFFFF)], 1)
    b, _, _ = p.run(torch, 0.125)
    np.testing.assert_array_equal(a, b)


def test_masked_tokens_do_not_leak(torch):
    """The value of a token that a row's mask hides has no effect on that row, however large."""
    rng = np.random.default_rng(7)
    p = H.Paged(rng, [20], [4], 2, 1, 64, 16, "bf16", tree=H.tree_of(max_back=1))
    p.mask[:, 0] = [1, 3, 1 | 4, 3 | 8]                  # row 2 does not see token 1
    a, _, _ = p.run(torch, 0.125)
    (c0, _), (s0, _), (v0, _), (w0, _) = S.block_parts(64)
    blk = p.cache[p.table[0, 1], 0, 0]                   # token 17 = new token 1
    blk[v0 + 32:v0 + 64], blk[w0 + 4:w0 + 8] = 0x77, 0x7E
    blk[c0 + 32:c0 + 64], blk[s0 + 4:s0 + 8] = 0x77, 0x7E
    b, _, _ = p.run(torch, 0.125)
    np.testing.assert_array_equal(a[[0, 2]], b[[0, 2]])
    assert (a[1] != b[1]).any()


@pytest.mark.parametrize("Ls", [[5000], [1, 4999, 3], [2000, 1, 700, 16, 1300, 47], [60000, 12]])
def test_long_and_ragged_lengths(torch, Ls):
    rng = np.random.default_rng(len(Ls))
    p = H.Paged(rng, Ls, [min(3, L) for L in Ls], 8, 2, 64, 128, "bf16")
    check(torch, p)


def test_many_requests(torch):
    rng = np.random.default_rng(11)
    lens = rng.integers(1, 70, 700)
    check(torch, H.Paged(rng, lens, np.minimum(lens, rng.integers(0, 4, 700)), 2, 1, 64, 16, "bf16"))


def test_requests_without_rows_or_tokens(torch):
    rng = np.random.default_rng(12)
    check(torch, H.Paged(rng, [0, 30, 0, 17, 50], [0, 2, 0, 0, 1], 4, 2, 64, 16, "bf16"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(torch, dtype):
    """Scores of hundreds, growing along the context: the running maximum has to follow."""
    rng = np.random.default_rng(13)
    p = H.Paged(rng, [700], [2], 4, 2, 128, 64, dtype, q_size=8.0)
    for i, t in enumerate(range(0, 700, 16)):            # scales grow with the position
        blk = p.cache[p.table[0, t // 64], :, t % 64 // 16]
        blk[:, 8 * 128:9 * 128] = 0x28 + i
    check(torch, p, scale=0.2)


def test_small_and_large_queries(torch):
    """Rows of very different size in one tile keep their own precision."""
    rng = np.random.default_rng(14)
    p = H.Paged(rng, [100], [6], 2, 1, 64, 16, "f32")
    p.q *= (10.0 ** np.array([-30, -8, 0, 3, 12, 25]))[:, None, None]
    p.q = H.rounded(p.q, "f32")
    scale = 1e-3
    out, lse, st = p.run(torch, scale)
    want, wlse, tol_o, tol_l = p.oracle(scale)
    assert st == 0
    near = tol_l < 0.1                                   # beyond it scores carry no digits
    assert near[:4].all()
    assert (np.abs(out - want) <= tol_o)[near].all()
    assert (np.abs(lse - wlse) <= tol_l)[near].all()


def test_query_strides_and_padding_rows(torch):
    """q is a slice of a wider projection; rows outside row_ptr are not touched."""
    rng = np.random.default_rng(15)
    p = H.Paged(rng, [50, 60], [3, 2], 4, 2, 64, 16, "bf16")
    wide = torch.randn((p.T + 4, 8, 64), device="cuda").to(torch.bfloat16)
    wide[2:2 + p.T, 1:5] = H.dev(p.q, torch.bfloat16)
    wide[:2] = float("nan")
    out, lse, st = p.run(torch, 0.125, q=wide[:, 1:5], row_ptr=H.dev(p.ptr + 2))
    want, _, tol, _ = p.oracle(0.125)
    assert st == 0 and (np.abs(out[2:7] - want) <= tol).all()
    assert (out[:2] == 7).all() and (out[7:] == 7).all() and (lse[:2] == 7).all()


def test_negative_scale_and_no_lse(torch):
    rng = np.random.default_rng(16)
    check(torch, H.Paged(rng, [77], [3], 4, 2, 64, 16, "bf16"), scale=-0.1, lse=False)


def test_repeatable_and_on_another_stream(torch):
    rng = np.random.default_rng(17)
    p = H.Paged(rng, rng.integers(200, 3000, 9), [4] * 9, 8, 2, 128, 64, "bf16")
    a = p.run(torch, 0.09)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b = p.run(torch, 0.09)
    c = p.run(torch, 0.09, stream=s)
    for x in (b, c):
        np.testing.assert_array_equal(a[0], x[0])
        np.testing.assert_array_equal(a[1], x[1])


def test_captured_in_a_graph(torch):
    L = H.lib()
    rng = np.random.default_rng(18)
    p = H.Paged(rng, [90, 400], [2, 3], 8, 2, 64, 64, "bf16")
    want, _, _ = p.run(torch, 0.125)
    q, cache, table = H.dev(p.q, torch.bfloat16), H.dev(p.cache), H.dev(p.table)
    lens, ptr, st = H.dev(p.lens), H.dev(p.ptr), H.new_status()
    out = torch.zeros_like(q)
    ws = torch.empty(L.spec_cache_attention_workspace_bytes(8, 2, 64), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        L.spec_cache_attention(q, cache, table, lens, ptr, out, st, ws, 0.125, p.k_scale, p.v_scale)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        L.spec_cache_attention(q, cache, table, lens, ptr, out, st, ws, 0.125, p.k_scale, p.v_scale)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(out.double().cpu().numpy(), want)


def test_pages_beyond_2_to_the_32_bytes(torch):
    """A cache of more than 4 GB, the request's pages at its end."""
    rng = np.random.default_rng(19)
    p = H.Paged(rng, [300], [2], 4, 2, 128, 128, "bf16", extra_pages=0)
    small = p.cache
    per = small[0].nbytes
    far = (9 << 30) // per
    big = torch.zeros((far + len(small), *small.shape[1:]), dtype=torch.uint8, device="cuda")
    big[far:] = H.dev(small)
    L = H.lib()
    q, st = H.dev(p.q, torch.bfloat16), H.new_status()
    out = torch.empty_like(q)
    ws = torch.empty(L.spec_cache_attention_workspace_bytes(4, 2, 128), dtype=torch.uint8, device="cuda")
    table = H.dev(np.where(p.table >= 0, p.table + far, -1).astype(np.int32))
    L.spec_cache_attention(q, big, table, H.dev(p.lens), H.dev(p.ptr), out, st, ws, 0.1, p.k_scale, p.v_scale)
    torch.cuda.synchronize()
    want, _, tol, _ = p.oracle(0.1)
    assert H.status(st) == 0 and (np.abs(out.double().cpu().numpy() - want) <= tol).all()


def test_bad_requests_get_nan_and_leave_the_others(torch):
    rng = np.random.default_rng(20)
    p = H.Paged(rng, [40, 50, 60, 700], [2, 2, 2, 2], 4, 2, 64, 16, "bf16")
    want, _, tol, _ = p.oracle(0.125)
    p.lens[1] = 1                                        # below its rows
    p.table[2, 1] = 10 ** 6                              # a page outside the cache
    p.lens[0] = 16 * p.table.shape[1] + 1                # more tokens than table entries
    out, lse, st = p.run(torch, 0.125)
    assert st == BAD_LEN | BAD_SLOT
    assert np.isnan(out[:6]).all() and np.isnan(lse[:6]).all()
    assert (np.abs(out[6:] - want[6:]) <= tol[6:]).all()


def test_row_ptr_out_of_range(torch):
    rng = np.random.default_rng(21)
    p = H.Paged(rng, [40, 50], [2, 2], 4, 2, 64, 16, "bf16")
    want, _, tol, _ = p.oracle(0.125)
    for ptr in ([0, 2, 9], [-3, 2, 4]):
        out, _, st = p.run(torch, 0.125, row_ptr=H.dev(np.array(ptr, np.int32)))
        assert st & BAD_LEN


def test_nan_query_stays_in_its_row(torch):
    rng = np.random.default_rng(22)
    p = H.Paged(rng, [80], [4], 4, 2, 64, 16, "bf16")
    want, _, tol, _ = p.oracle(0.125)
    q = p.q.copy()
    q[1, 2, 5] = np.nan
    out, lse, _ = p.run(torch, 0.125, q=H.dev(q, torch.bfloat16))
    assert np.isnan(out[1, 2]).all() and np.isnan(lse[1, 2])
    keep = np.ones(out.shape[:2], bool)
    keep[1, 2] = False
    assert (np.abs(out - want) <= tol)[keep].all()


# heads of 128 elements with more rows than one tile, and with rows that fill a wide tile
@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 5), (8, 1, 4), (4, 1, 8), (6, 2, 7), (32, 8, 8), (16, 2, 9), (24, 1, 3)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_wide_row_tiles(torch, Hq, Hkv, n, page):
    rng = np.random.default_rng(Hq * n + page)
    lens = [n, n + 1, 127, 128, 129, 255, 300, 1000]
    check(torch, H.Paged(rng, lens, [n] * 8, Hq, Hkv, 128, page, "bf16"))


@pytest.mark.parametrize("n", [9, 25, 40, 70])
@pytest.mark.parametrize("empty", [False, True])
def test_wide_tree_masks(torch, n, empty):
    rng = np.random.default_rng(n)
    p = H.Paged(rng, [n, n + 1, n + 100, n + 500, n + 128], [n] * 5, 4, 1, 128, 32, "bf16", tree=H.tree_of(empty=empty))
    out, lse = check(torch, p)
    assert not empty or ((out[n // 2] == 0).all() and np.isneginf(lse[n // 2]).all())


def test_wide_ragged_rows_and_long_lengths(torch):
    rng = np.random.default_rng(31)
    lens = [20000, 5, 300, 1, 2500, 640, 77]
    check(torch, H.Paged(rng, lens, [8, 2, 0, 1, 17, 3, 40], 8, 2, 128, 64, "bf16"))


def test_wide_large_scores(torch):
    """A 16-bit float ends at 2^-24: with the row's largest p at 2^7 or more, p below 2^-21 of it
    are off by up to 2^-32 of it, which shows in an element to which the largest p add zeros."""
    rng = np.random.default_rng(32)
    p = H.Paged(rng, [900, 300], [6, 3], 8, 1, 128, 64, "bf16", q_size=8.0)
    for i, t in enumerate(range(0, 900, 16)):
        blk = p.cache[p.table[0, t // 64], :, t % 64 // 16]
        blk[:, 8 * 128:9 * 128] = 0x28 + min(i, 0x55)
    floor = 2.0 ** -32 * 900 * 6 * 2.0 ** 6 * p.v_scale      # of the tokens' sum of |v|
    for scale in (0.2, -0.2, 0.0):
        check(torch, p, scale=scale, floor=floor)


def test_wide_query_strides_and_padding_rows(torch):
    rng = np.random.default_rng(35)
    p = H.Paged(rng, [900, 300], [6, 3], 8, 1, 128, 64, "bf16")
    wide = torch.randn((p.T + 4, 10, 128), device="cuda").to(torch.bfloat16)
    wide[2:2 + p.T, 1:9] = H.dev(p.q, torch.bfloat16)
    out, lse, st = p.run(torch, 0.1, q=wide[:, 1:9], row_ptr=H.dev(p.ptr + 2))
    want, _, tol, _ = p.oracle(0.1)
    assert st == 0 and (np.abs(out[2:11] - want) <= tol).all()
    assert (out[:2] == 7).all() and (out[11:] == 7).all() and (lse[11:] == 7).all()


def test_wide_bad_requests(torch):
    rng = np.random.default_rng(33)
    p = H.Paged(rng, [400, 500, 600, 700, 300], [5] * 5, 8, 2, 128, 64, "bf16")
    want, _, tol, _ = p.oracle(0.1)
    p.lens[1] = 1
    p.table[2, 1] = -5
    p.lens[0] = 64 * p.table.shape[1] + 1
    out, lse, st = p.run(torch, 0.1)
    assert st == BAD_LEN | BAD_SLOT
    assert np.isnan(out[:15]).all() and np.isnan(lse[:15]).all()
    assert (np.abs(out[15:] - want[15:]) <= tol[15:]).all()


def test_wide_nan_query_and_repeats(torch):
    rng = np.random.default_rng(34)
    p = H.Paged(rng, rng.integers(100, 3000, 12), [6] * 12, 8, 2, 128, 16, "bf16")
    want, _, tol, _ = p.oracle(0.1)
    a = p.run(torch, 0.1)
    for _ in range(3):
        b = p.run(torch, 0.1, stream=torch.cuda.Stream())
        np.testing.assert_array_equal(a[0], b[0])
        np.testing.assert_array_equal(a[1], b[1])
    q = p.q.copy()
    q[7, 3, 9], q[20, 0, 100] = np.nan, np.inf
    out, lse, _ = p.run(torch, 0.1, q=H.dev(q, torch.bfloat16))
    bad = np.zeros(out.shape[:2], bool)
    bad[7, 3] = bad[20, 0] = True
    assert np.isnan(out[bad]).all()
    assert (np.abs(out - want) <= tol)[~bad].all()
