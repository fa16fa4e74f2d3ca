"""A tree between chains on the paged cache, the way the header describes it: its rows see their
ancestors, nothing of its block is kept, and the next block begins with the accepted path's tokens;
attention then sees the context, the path and the block, and no rejected node."""
import numpy as np
import pytest

from oracle import serving as S
from tests import serving as H

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE = 4, 2, 64, 16
G = (0.00893, 0.00227)


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def test_a_tree_and_the_block_after_it(torch):
    from speculative_decoding_draft_04_gb300 import engine
    rng = np.random.default_rng(8)
    prompts, N, n = np.array([21, 9]), 12, 4
    # the accepted path's rows of each tree's block (row 0: the anchor)
    paths = [[0, 2, 7], [0, 1, 3, 8, 11]]
    parents = []
    for path in paths:
        parent = [-1] + [int(rng.integers(0, i)) for i in range(1, N)]
        for a, b in zip(path, path[1:]):
            parent[b] = a
        parents.append(parent)
    mask = np.zeros((2 * N, 1), np.uint32)
    for b, parent in enumerate(parents):
        for i in range(N):
            mask[b * N + i] = (mask[b * N + parent[i]] if i else 0) | np.uint32(1 << i)
    c = engine.DeviceCache.allocate(2, 1, HQ, HKV, D, PAGE, 8, 64, 64, [G[0]], [G[1]])
    kept = [[np.zeros((0, HKV, D)) for _ in range(2)] for _ in range(2)]     # [which][request]

    def step(accept, keep, k, v, bits=None):
        """A block of rows k, v per request: the kept tokens are the first keep[b]."""
        count = [len(x) for x in k]
        engine.make_room(c, H.dev(np.array(count, np.int32)),
                         None if accept is None else H.dev(np.array(accept, np.int32)))
        q = [rng.normal(size=(m, HQ, D)).astype(np.float32) for m in count]
        out = torch.empty((sum(count), HQ, D), dtype=torch.float32, device="cuda")
        engine.attend(c, 0, H.dev(np.concatenate(q)), H.dev(np.concatenate(k)), H.dev(np.concatenate(v)), out,
                      tree_mask=None if bits is None else H.dev(bits.view(np.int32)))
        out = out.double().cpu().numpy()
        at = 0
        for b, m in enumerate(count):
            for which, x in enumerate((k[b], v[b])):
                g = np.float64(np.float32(G[which]))
                code, s = S.store(x.reshape(-1, 16), g)
                kept[which][b] = np.concatenate([kept[which][b][:keep[b]], S.values(code, s, g).reshape(m, HKV, D)])
            see = S.visible(m, len(kept[0][b]), None if bits is None else bits[at:at + m])
            for h in range(HQ):
                kk, vv = (kept[x][b][:, h * HKV // HQ] for x in (0, 1))
                o, _, absv, big = S.attention(q[b][:, h].astype(np.float64), kk, vv, see, D ** -0.5)
                tol = 2.0 ** -22 * np.abs(o) + (2.0 ** -20 + 2.0 ** -17 * big[:, None] + 2.0 ** -15) * absv + 1e-30
                assert (np.abs(out[at:at + m, h] - o) <= tol).all(), (b, h)
            at += m
        assert c.kv_len.cpu().tolist() == [len(x) for x in kept[0]]

    def rows(*count):
        return [rng.normal(size=(m, HKV, D)).astype(np.float32) for m in count]
    step(None, [0, 0], rows(*prompts), rows(*prompts))
    tk, tv = rows(N, N), rows(N, N)
    step(prompts - 1, prompts, tk, tv, mask)
    more_k, more_v = rows(n, n), rows(n, n)
    step([-1, -1], prompts, [np.concatenate([tk[b][paths[b]], more_k[b]]) for b in range(2)],
         [np.concatenate([tv[b][paths[b]], more_v[b]]) for b in range(2)])
    held = prompts + [len(p) for p in paths] + 2             # two of the block after the path
    step([len(p) + 1 for p in paths], held, rows(n, n), rows(n, n))
    assert c.seq_len[c.newest].cpu().tolist() == held.tolist()
    assert engine.status_words(c.status)[0] == 0
