"""GPU parity of spec_cache_attention where requests have more than 32 rows a
key-value head (trees, prompts; tiles of 128 rows): tile edges, ragged rows,
pages that end inside a unit, split and many short requests, masks, strides,
rows that see nothing, refused pages and lengths.  Tolerances:
test_cache_attention_gpu.py."""
import numpy as np
import pytest

import serving as H
from test_cache_attention_gpu import BAD_LEN, BAD_SLOT, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 1, 9), (8, 2, 32), (8, 2, 33), (2, 2, 127), (2, 2, 128), (3, 1, 43),
                                      (40, 1, 4), (2, 1, 130)])
def test_tile_edges(torch, D, Hq, Hkv, n):
    rng = np.random.default_rng(D + Hq * n)
    page = (16, 32, 64, 128)[n % 4]
    lens = [n, n + 1, n + 63, 2 * n + 64, n + 200]
    check(torch, H.Paged(rng, lens, [n] * 5, Hq, Hkv, D, page, "bf16"))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_trees_and_ragged_rows(torch, page):
    rng = np.random.default_rng(page)
    news = [25, 1, 60, 0, 33, 64, 2, 48]
    lens = [n + int(rng.integers(0, 300)) for n in news]
    check(torch, H.Paged(rng, lens, news, 8, 2, 128, page, "bf16", tree=H.tree_of(empty=True)))
    check(torch, H.Paged(rng, lens, news, 8, 2, 64, page, "bf16", tree=H.tree_of()))


def test_split_requests(torch):
    """Few requests over many units: parts joined across CTAs, rows of a second tile."""
    rng = np.random.default_rng(3)
    check(torch, H.Paged(rng, [4097, 9000], [35, 70], 4, 1, 128, 64, "bf16"))


def test_many_short_requests(torch):
    """Several segments a CTA, one or two units each."""
    rng = np.random.default_rng(4)
    lens = rng.integers(40, 70, 150)
    check(torch, H.Paged(rng, lens, [40] * 150, 4, 4, 64, 16, "bf16"))


def test_prompt_without_context(torch):
    rng = np.random.default_rng(5)
    check(torch, H.Paged(rng, [300, 257], [300, 257], 4, 2, 128, 32, "bf16"))


@pytest.mark.parametrize("scale", [0.2, -0.2, 0.0])
def test_growing_scores(torch, scale):
    """The running maximum has to follow; the floor is the 16-bit float's least step (2^-32 of a row's
    largest p) of the tokens' sum of |v|."""
    rng = np.random.default_rng(6)
    p = H.Paged(rng, [900, 300], [50, 41], 8, 4, 128, 64, "bf16", q_size=8.0)
    for i, t in enumerate(range(0, 900, 16)):
        blk = p.cache[p.table[0, t // 64], :, t % 64 // 16]
        blk[:, 8 * 128:9 * 128] = 0x28 + min(i, 0x55)
    check(torch, p, scale=scale, floor=2.0 ** -32 * 900 * 6 * 2.0 ** 6 * p.v_scale)


def test_small_queries(torch):
    rng = np.random.default_rng(10)
    p = H.Paged(rng, [100, 90], [36, 40], 2, 1, 64, 16, "bf16")
    p.q = H.rounded(p.q * (10.0 ** rng.integers(-30, 1, (p.T, 1, 1))), "bf16")
    check(torch, p)


def test_pages_outside_the_cache(torch):
    rng = np.random.default_rng(7)
    p = H.Paged(rng, [200, 300, 250], [40, 40, 40], 4, 2, 128, 16, "bf16")
    want, _, tol, _ = p.oracle(0.1)
    p.table[1, 3] = 10 ** 6
    out, l, st = p.run(torch, 0.1)
    assert st == BAD_SLOT
    for b in (0, 2):
        r = slice(p.ptr[b], p.ptr[b + 1])
        assert (np.abs(out[r] - want[r]) <= tol[r]).all()
    assert np.isnan(out[p.ptr[1]:p.ptr[2]]).all() and np.isnan(l[p.ptr[1]:p.ptr[2]]).all()


def test_lengths_outside_the_table(torch):
    rng = np.random.default_rng(8)
    p = H.Paged(rng, [200, 300, 250], [40, 40, 40], 4, 2, 64, 16, "bf16")
    want, _, tol, _ = p.oracle(0.1)
    p.lens[0], p.lens[1] = 39, 10 ** 9                     # below its rows; beyond its pages
    out, l, st = p.run(torch, 0.1)
    assert st == BAD_LEN
    assert np.isnan(out[:80]).all() and np.isnan(l[:80]).all()
    assert (np.abs(out[80:] - want[80:]) <= tol[80:]).all()


def test_strides_streams_and_repeats(torch):
    rng = np.random.default_rng(9)
    p = H.Paged(rng, [700, 900, 64], [64, 40, 50], 8, 2, 128, 64, "bf16", tree=H.tree_of())
    wide = torch.zeros((p.T + 5, 3, 8, 128), dtype=torch.bfloat16, device="cuda")
    wide[:p.T, 1] = H.dev(p.q, torch.bfloat16)
    wide[p.T:] = float("nan")                              # rows of no request
    want, lse, tol_o, tol_l = p.oracle(0.09)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = None
    mask = p.mask
    p.mask = np.concatenate([mask, np.zeros((5, mask.shape[1]), np.uint32)])
    for _ in range(3):
        out, l, st = p.run(torch, 0.09, stream=side, q=wide[:, 1])
        assert st == 0 and (out[p.T:] == 7).all() and (l[p.T:] == 7).all()
        assert (np.abs(out[:p.T] - want) <= tol_o).all()
        assert (np.abs(l[:p.T] - lse) <= tol_l).all()
        assert first is None or (out == first).all()       # bit for bit
        first = out


def test_offsets_beyond_2_to_the_32(torch):
    rng = np.random.default_rng(11)
    p = H.Paged(rng, [90, 200], [36, 50], 4, 2, 128, 64, "bf16")
    small = p.cache
    per = int(np.prod(small.shape[1:]))
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
