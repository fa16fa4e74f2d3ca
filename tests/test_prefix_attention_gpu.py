"""Attention with shared prefixes (spec_prefix_attention) against the float64 oracle over prefix and own
tokens together, which reads the same bytes.  Tolerances as in test_cache_attention_gpu: the two parts'
sums are joined by factors 2^(m - max) exact to 2^-22 and one rounding more, inside the 2^-15 of
sum p |v| (and the 2^-20 of lse) there."""
import numpy as np
import pytest

from oracle import serving as S
from tests import serving as H

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


class Shared:
    """Requests of groups behind prefixes, all in one random cache."""

    def __init__(self, rng, groups, prefixes, lens, news, Hq, Hkv, D, page, dtype, tree=None):
        self.groups, self.prefixes = list(groups), list(prefixes)
        self.B = sum(groups)
        n = len(prefixes)
        # the prefixes are further "requests" without new rows
        self.p = H.Paged(rng, list(lens) + list(prefixes), list(news) + [0] * n, Hq, Hkv, D, page, dtype, tree=tree)
        self.cut = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)

    def run(self, torch, stream=None, **change):
        p, L = self.p, H.lib()
        a = dict(table=p.table[:self.B], lens=p.lens[:self.B], ptr=p.ptr[:self.B + 1], ptable=p.table[self.B:],
                 plen=p.lens[self.B:], cut=self.cut, q=H.dev(p.q, H.storage(torch, p.dtype)))
        a.update(change)
        T = a["q"].shape[0]
        st = H.new_status()
        out = torch.full((T, p.Hq, p.D), 7.0, dtype=H.storage(torch, p.dtype), device="cuda")
        lse = torch.full((T, p.Hq), 7.0, device="cuda")
        ws = torch.full((L.spec_prefix_attention_workspace_bytes(T, p.Hq, p.Hkv, p.D),), 0xA5, dtype=torch.uint8,
                        device="cuda")
        L.spec_prefix_attention(a["q"], H.dev(p.cache), H.dev(a["table"]), H.dev(a["lens"]), H.dev(a["ptr"]),
                                H.dev(a["ptable"]), H.dev(a["plen"]), H.dev(a["cut"]), out, st, ws, p.D ** -0.5,
                                p.k_scale, p.v_scale,
                                tree_mask=None if p.mask is None else H.dev(p.mask.view(np.int32)), lse=lse, stream=stream)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), lse.double().cpu().numpy(), H.status(st)

    def oracle(self):
        p, G = self.p, self.p.Hq // self.p.Hkv
        out, lse = np.zeros((p.T, p.Hq, p.D)), np.zeros((p.T, p.Hq))
        tol_o, tol_l = np.zeros_like(out), np.zeros_like(lse)
        half = 2.0 ** -8 if p.dtype == "bf16" else 2.0 ** -22
        prob = 2.0 ** -11 if p.dtype == "bf16" else 2.0 ** -20
        group = np.repeat(np.arange(len(self.groups)), self.groups)
        for b in range(self.B):
            n, L, F = int(p.news[b]), int(p.lens[b]), int(self.prefixes[group[b]])
            r = slice(p.ptr[b], p.ptr[b + 1])
            see = np.concatenate([np.ones((n, F), bool), S.visible(n, L, None if p.mask is None else p.mask[r])], 1)
            for h in range(p.Hkv):
                k, v = (np.concatenate([S.read_tokens(p.cache, p.table[self.B + group[b]], h, F, p.D, i, g),
                                        S.read_tokens(p.cache, p.table[b], h, L, p.D, i, g)])
                        for i, g in ((0, p.k_scale), (1, p.v_scale)))
                for i in range(h * G, (h + 1) * G):
                    o, l, absv, big = S.attention(p.q[r, i], k, v, see, p.D ** -0.5)
                    out[r, i], lse[r, i] = o, l
                    x = 2.0 ** -18 * big[:, None]
                    tol_o[r, i] = half * np.abs(o) + (prob + 2 * x + 2.0 ** -15) * absv + 1e-30
                    tol_l[r, i] = x[:, 0] + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(l), l, 0)))
        return out, lse, tol_o, tol_l


def tree_of(rng, p):
    """Ancestor masks of random trees over the new rows of the requests that have some; one row of
    each sees nothing."""
    mask = np.zeros((p.T, -(-int(p.news.max()) // 32)), np.uint32)
    for first, n in zip(p.ptr[:-1], p.news):
        for i in range(n):
            if i:
                mask[first + i] = mask[first + rng.integers(max(0, i - 4), i)]
            mask[first + i, i // 32] |= np.uint32(1 << (i % 32))
        if n:
            mask[first + n // 2] = 0
    return mask


def check(torch, s, **kw):
    out, lse, st = s.run(torch, **kw)
    want, wlse, tol_o, tol_l = s.oracle()
    assert st == 0
    bad = ~(np.abs(out - want) <= tol_o)
    assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5], want[bad][:5], tol_o[bad][:5])
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
    check(torch, Shared(rng, [3, 1, 2], [130, 0, 77], [1, 17, 64, 40, 90, 8], [1, 1, 3, 2, 8, 8], 6, 2, D, page, dtype))


@pytest.mark.parametrize("F", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("rows", [1, 40])
def test_prefix_lengths(torch, F, rows):
    """Few rows a group (tiles of 8) and many (tiles of 128)."""
    rng = np.random.default_rng(F)
    check(torch, Shared(rng, [rows], [F], rng.integers(1, 50, rows), [1] * rows, 4, 1, 64, 32, "bf16"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("groups,prefixes", [([5], [0]), ([2, 3], [0, 40]), ([0, 5], [40, 20]), ([1] * 5, [10, 20, 0, 30, 1]),
                                             ([4, 0, 1], [64, 0, 16])])
def test_groups(torch, dtype, groups, prefixes):
    rng = np.random.default_rng(sum(prefixes))
    check(torch, Shared(rng, groups, prefixes, [5, 30, 1, 64, 33], [2, 1, 1, 4, 3], 4, 2, 64, 16, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 3, 4, 8])
def test_many_rows_of_a_group(torch, dtype, G):
    """Groups of several row tiles, whose long prefix is shared out."""
    rng = np.random.default_rng(G)
    news = rng.integers(1, 9, 40)
    check(torch, Shared(rng, [37, 3], [900, 333], news + rng.integers(0, 40, 40), news, 2 * G, 2, 128, 64, dtype))


@pytest.mark.parametrize("n", [5, 25, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_trees_and_rows_that_see_nothing_of_their_own(torch, n, dtype):
    rng = np.random.default_rng(n)
    s = Shared(rng, [2, 2], [100, 0], [n, n + 30, n, n + 3], [n] * 4, 4, 1, 64, 32, dtype, tree=tree_of)
    out, lse = check(torch, s)
    nothing = s.p.ptr[2] + n // 2                            # no prefix, no context, no bit
    assert (out[nothing] == 0).all() and np.isneginf(lse[nothing]).all()


def test_the_same_numbers_as_whole_tables(torch):
    """Prefix and own tokens in one table, by spec_cache_attention: as far apart as two calls may be."""
    rng = np.random.default_rng(7)
    s = Shared(rng, [6], [128], rng.integers(1, 60, 6), [1] * 6, 8, 2, 128, 32, "bf16")
    out, lse, _ = s.run(torch)
    p = s.p
    whole = H.Paged.__new__(H.Paged)
    whole.__dict__.update(p.__dict__)
    whole.lens, whole.news = (p.lens[:6] + 128).astype(np.int32), p.news[:6]
    whole.table = np.concatenate([np.repeat(p.table[6:, :4], 6, 0), p.table[:6]], 1)
    whole.ptr = p.ptr[:7]
    o2, l2, st = whole.run(torch, 128 ** -0.5)
    want, wlse, tol_o, tol_l = s.oracle()
    assert st == 0 and (np.abs(out - o2) <= 2 * tol_o).all() and (np.abs(lse - l2) <= 2 * tol_l).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f32", 64), ("bf16", 256)])
def test_bad_prefixes(torch, dtype, D):
    rng = np.random.default_rng(2)
    s = Shared(rng, [20, 3], [100, 40], [9] * 23, [1] * 23, 4, 2, D, 16, dtype)
    good, _, _ = s.run(torch)
    for length in (-1, 16 * s.p.table.shape[1] + 1, 2 ** 31 - 1):
        plen = np.array([100, length], np.int32)
        out, lse, st = s.run(torch, plen=plen)
        assert st == BAD_LEN and np.isnan(out[20:]).all() and np.isnan(lse[20:]).all()
        assert np.array_equal(out[:20], good[:20])
    for page in (-1, len(s.p.cache)):
        table = s.p.table[23:].copy()
        table[0, 2] = page
        out, lse, st = s.run(torch, ptable=table)
        assert st == BAD_SLOT and np.isnan(out[:20]).all() and np.array_equal(out[20:], good[20:])
    lens = s.p.lens[:23].copy()
    lens[4] = 0                                              # fewer tokens than rows
    out, _, st = s.run(torch, lens=lens)
    assert st == BAD_LEN and np.isnan(out[4]).all()
    keep = np.arange(23) != 4
    assert np.array_equal(out[keep], good[keep])


@pytest.mark.parametrize("cut", [[0, 20, 22], [1, 20, 23], [0, 24, 23], [0, -1, 23], [0, 20, 2 ** 31 - 1]])
def test_groups_that_are_no_partition(torch, cut):
    rng = np.random.default_rng(3)
    s = Shared(rng, [20, 3], [100, 40], [9] * 23, [1] * 23, 4, 2, 64, 16, "bf16")
    out, lse, st = s.run(torch, cut=np.array(cut, np.int32))
    assert st == BAD_LEN and np.isnan(out).all() and np.isnan(lse).all()


def test_rows_of_no_request_are_left(torch):
    rng = np.random.default_rng(4)
    s = Shared(rng, [5], [50], [9] * 5, [1] * 5, 4, 2, 64, 16, "bf16")
    q = torch.cat([H.dev(s.p.q, torch.bfloat16), torch.full((60, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out, lse, st = s.run(torch, q=q)
    want, _, tol, _ = s.oracle()
    assert st == 0 and (np.abs(out[:5] - want) <= tol).all() and (out[5:] == 7).all() and (lse[5:] == 7).all()


def test_captured_and_on_two_streams(torch):
    rng = np.random.default_rng(5)
    s = Shared(rng, [30, 2], [700, 64], rng.integers(2, 80, 32), [2] * 32, 8, 2, 128, 32, "bf16")
    p, L = s.p, H.lib()
    args = [H.dev(x) for x in (p.cache, p.table[:32], p.lens[:32], p.ptr[:33], p.table[32:], p.lens[32:], s.cut)]
    q, st = H.dev(p.q, torch.bfloat16), H.new_status()
    outs = [torch.zeros_like(q) for _ in range(3)]
    ws = [torch.empty(L.spec_prefix_attention_workspace_bytes(p.T, 8, 2, 128), dtype=torch.uint8, device="cuda")
          for _ in range(3)]

    def call(i, stream=None):
        L.spec_prefix_attention(q, *args, outs[i], st, ws[i], 128 ** -0.5, p.k_scale, p.v_scale, stream=stream)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):                                       # at once, each in its workspace
        call(0)
        call(1, other)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(2)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and H.status(st) == 0
