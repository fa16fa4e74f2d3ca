"""A server's steps with the operators together: instructions that groups of requests share go into
the cache once, each request appends its own prompt, its first token is drawn, and decoding goes on --
queries and keys normed and rotated by positions that count the prefix, attention over prefix and own
tokens, a token drawn from each request's logits."""
import numpy as np
import pytest

from oracle import serving as S
from tests import serving as H

pytestmark = pytest.mark.gpu
HQ, HKV, D, PAGE, LAYERS = 8, 2, 64, 16, 2
K_SCALE, V_SCALE = [0.0121, 0.0101], [0.0027, 0.0031]


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def test_decoding_behind_shared_prefixes(torch):
    from speculative_decoding_draft_04_gb300 import _lib, engine
    rng = np.random.default_rng(21)
    sizes, prefix, prompts = [3, 2], [37, 16], np.array([5, 16, 1, 20, 9])
    B, groups, V = 5, 2, 3000
    c = engine.DeviceCache.allocate(B + groups, LAYERS, HQ, HKV, D, PAGE, 40, 80, 60, K_SCALE, V_SCALE)
    s = engine.Prefixes.allocate(c, sizes, HQ)
    with pytest.raises(_lib.SpecError):
        engine.Prefixes.allocate(c, [5, 2], HQ)
    qw, kw = ([H.dev(rng.normal(1, 0.2, D).astype(np.float32)) for _ in range(LAYERS)] for _ in range(2))
    rotary = engine.Rotary.table(128, D, q_weight=qw, k_weight=kw)
    rope = rotary.rope.cpu().numpy()
    group = np.repeat(np.arange(groups), sizes)
    held = [[[np.zeros((0, HKV, D)) for _ in range(B + groups)] for _ in range(2)] for _ in range(LAYERS)]
    g = [[np.float64(np.float32(x)) for x in y] for y in (K_SCALE, V_SCALE)]

    def attend(count, prefixes):
        """Random rows of every layer, checked against everything held so far."""
        ptr = np.concatenate([[0], np.cumsum(count)])
        T = int(ptr[-1])
        who = np.repeat(np.arange(B + groups), count)
        for layer in range(LAYERS):
            q, k, v = (rng.normal(size=(T, h, D)).astype(np.float32) for h in (HQ, HKV, HKV))
            before = [len(x) for x in held[layer][0]]
            at = np.concatenate([np.arange(n) + before[i] + (before[B + group[i]] if i < B else 0)
                                 for i, n in enumerate(count)])
            out = torch.empty((T, HQ, D), dtype=torch.float32, device="cuda")
            engine.attend(c, layer, H.dev(q), H.dev(k), H.dev(v), out, rotary=rotary, prefixes=prefixes)
            if prefixes is not None:
                assert prefixes.positions.cpu().tolist()[:T] == at.tolist()
            q = S.rotated(q, rope[at], qw[layer].cpu().numpy())
            k = S.rotated(k, rope[at], kw[layer].cpu().numpy())
            for which, x in enumerate((k, v)):
                code, sc = S.store(x.reshape(-1, 16), g[which][layer])
                x = S.values(code, sc, g[which][layer]).reshape(T, HKV, D)
                for i in range(B + groups):
                    held[layer][which][i] = np.concatenate([held[layer][which][i], x[who == i]])
            out = out.double().cpu().numpy()
            for i in range(B + groups):
                n = int(count[i])
                if n == 0:
                    continue
                F = before[B + group[i]] if i < B else 0
                L = len(held[layer][0][i])
                see = np.concatenate([np.ones((n, F), bool), S.visible(n, L)], 1)
                for h in range(HQ):
                    kk, vv = (held[layer][x][i][:, h * HKV // HQ] for x in (0, 1))
                    if F:
                        kk, vv = (np.concatenate([held[layer][x][B + group[i]][:, h * HKV // HQ], y])
                                  for x, y in ((0, kk), (1, vv)))
                    o, _, absv, big = S.attention(q[ptr[i]:ptr[i + 1], h].astype(np.float64), kk, vv, see, D ** -0.5)
                    x = 2.0 ** -18 * big[:, None]
                    tol = 2.0 ** -22 * np.abs(o) + (2.0 ** -20 + 2 * x + 2.0 ** -15) * absv + 1e-30
                    assert (np.abs(out[ptr[i]:ptr[i + 1], h] - o) <= tol).all(), (layer, i, h)

    # the holders' prompts, then the requests'
    count = np.array([0] * B + prefix)
    engine.make_room(c, H.dev(count.astype(np.int32)))
    attend(count, None)
    kept = np.array([-1] * B + [n - 1 for n in prefix], np.int32)
    drawn = engine.DeviceSampling.allocate(B, top_k=40, top_p=[0.9, 1.0, 0.5, 1.0, 0.95], min_p=0.001)
    step = np.concatenate([prompts, np.zeros(groups, np.int64)])
    for _ in range(4):
        engine.make_room(c, H.dev(step.astype(np.int32)), H.dev(kept))
        engine.place_after(c, s)
        attend(step, s)
        x = (rng.normal(size=(B, 1, V)) * 2).astype(np.float32)
        u, T = rng.random((B, 1)).astype(np.float32), np.full(B, 0.8, np.float32)
        engine.sample(H.dev(x), H.dev(u), H.dev(T), drawn)
        for b in range(B):
            p = [0.9, 1.0, 0.5, 1.0, 0.95][b]
            token, lp, n, near = S.sample(x[b, 0], float(T[b]), float(u[b, 0]), 40, float(np.float32(p)), float(np.float32(0.001)))
            assert near > 1e-9 and (int(drawn.tokens[b, 0]), int(drawn.kept[b, 0])) == (token, n)
            assert abs(float(drawn.logprob[b, 0]) - lp) <= 2.0 ** -23 * abs(lp) + 2.0 ** -31
        kept = np.concatenate([step[:B] - 1, [-1] * groups]).astype(np.int32)      # holders keep what they hold
        step = np.array([1] * B + [0] * groups)
    assert c.kv_len.cpu().tolist() == (prompts + 3).tolist() + prefix
    assert [engine.status_words(t)[0] for t in (c.status, drawn.status)] == [0, 0]
