"""The served cycle (draft, room in the paged cache, the target's pass over the
block, verify, log probabilities) over several cycles: lengths and pages follow
what each verification accepted, every layer's attention sees exactly the
tokens that were kept, and the reported log probabilities are those of the
emitted tokens.  And the example that runs it."""
import os
import runpy

import numpy as np
import pytest

from oracle import serving as S
from tests import serving as H

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE, LAYERS = 8, 2, 64, 16, 2
K_SCALE, V_SCALE = [0.00893, 0.0101], [0.00227, 0.0031]


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def test_cycles_keep_what_was_accepted(torch):
    from speculative_decoding_draft_04_gb300 import engine
    from speculative_decoding_draft_04_gb300 import workloads as W
    w = W.make_workload(W.config("C0", L=("uniform", 0, 4)), 3)
    d = engine.DeviceWorkload.from_workload(w)
    b = engine.Buffers.for_workload(d)
    B, n, V = w.B, w.gamma + 1, w.V
    prompts = np.array([1, 15, 16, 37], np.int32)
    news = (w.verify_len + 1).astype(np.int32)
    cycles, top = 4, 3
    c = engine.DeviceCache.allocate(B, LAYERS, HQ, HKV, D, PAGE, 32, 128, int(prompts.sum()) + B * n,
                                    K_SCALE, V_SCALE)
    l = engine.DeviceLogprobs.allocate(B, n, V, K=top)
    rng = np.random.default_rng(11)
    g = [[np.float64(np.float32(x)) for x in s] for s in (K_SCALE, V_SCALE)]
    # every request's keys and values as stored, [layer][which][b]: [tokens][Hkv][D]
    kept = [[[np.zeros((0, HKV, D)) for _ in range(B)] for _ in range(2)] for _ in range(LAYERS)]

    def attend(count):
        """Append and attend random rows in every layer; check them against the kept tokens."""
        ptr = np.concatenate([[0], np.cumsum(count)])
        T = int(ptr[-1])
        for layer in range(LAYERS):
            q, k, v = (rng.normal(size=(T, h, D)).astype(np.float32) for h in (HQ, HKV, HKV))
            out = torch.empty((T, HQ, D), dtype=torch.float32, device="cuda")
            engine.attend(c, layer, H.dev(q), H.dev(k), H.dev(v), out)
            for which, x in enumerate((k, v)):
                code, s = S.store(x.reshape(-1, 16), g[which][layer])
                x = S.values(code, s, g[which][layer]).reshape(T, HKV, D)
                for i in range(B):
                    kept[layer][which][i] = np.concatenate([kept[layer][which][i], x[ptr[i]:ptr[i + 1]]])
            out = out.double().cpu().numpy()
            for i in range(B):
                L = len(kept[layer][0][i])
                see = S.visible(int(count[i]), L)
                for h in range(HQ):
                    kk, vv = (kept[layer][x][i][:, h * HKV // HQ] for x in (0, 1))
                    o, _, absv, big = S.attention(q[ptr[i]:ptr[i + 1], h].astype(np.float64), kk, vv, see, D ** -0.5)
                    x = 2.0 ** -18 * big[:, None]
                    tol = 2.0 ** -22 * np.abs(o) + (2.0 ** -20 + 2 * x + 2.0 ** -15) * absv + 1e-30
                    assert (np.abs(out[ptr[i]:ptr[i + 1], h] - o) <= tol).all(), (layer, i, h)

    engine.make_room(c, H.dev(prompts))
    attend(prompts)
    last = prompts - 1                                       # kept beyond the first token of the last block
    base = np.zeros(B, np.int32)

    for _ in range(cycles):
        def target_pass(d_, b_, c_, stream):
            # the last block's tokens beyond the accepted ones are gone
            for layer in kept:
                for which in layer:
                    for i in range(B):
                        which[i] = which[i][:base[i] + last[i] + 1]
            attend(news)
        engine.served_cycle(d, b, c, l, target_pass, H.dev(news), H.dev(last.astype(np.int32)))
        base = base + last + 1
        assert c.seq_len[c.newest].cpu().tolist() == base.tolist()
        assert c.kv_len.cpu().tolist() == (base + news).tolist()
        assert c.num_blocks[c.newest].cpu().tolist() == (-(-(base + news) // PAGE)).tolist()
        head, tail = c.ring_pos[c.newest].cpu().tolist()
        assert tail - head == 32 - int((-(-(base + news) // PAGE)).sum())
        pos = c.positions.cpu().numpy()[:news.sum()]
        assert pos.tolist() == np.concatenate([np.arange(x, x + m) for x, m in zip(base, news)]).tolist()
        last = b.accept_len.cpu().numpy().astype(np.int32)
        tokens = b.out_tokens.cpu().numpy()
        lp, ent, ids = (t.cpu().numpy() for t in (l.logprob, l.entropy, l.top_ids))
        for i in range(B):
            assert (tokens[i, :last[i] + 1] >= 0).all() and (tokens[i, last[i] + 1:] == -1).all()
            for j in range(n):
                if tokens[i, j] < 0:
                    assert np.isnan(lp[i, j]) and np.isnan(ent[i, j]) and (ids[i, j] == -1).all()
                    continue
                x, T = w.row_f64("target", i, j), float(w.temperature[i])
                wl, we, wi, _, m2 = S.logprobs(x, T, int(tokens[i, j]), top)
                tol = 2.0 ** -21 * (3 + 2 * np.abs(x).max() / T + m2)
                assert abs(lp[i, j] - wl) <= tol + 2.0 ** -22 * abs(wl)
                assert abs(ent[i, j] - we) <= 2.0 ** -20 * (1 + we + m2) + tol
                assert ids[i, j].tolist() == wi.tolist()
        # other tokens in the next cycle
        d.u_draft.copy_(torch.from_numpy(W.uniforms(rng, (B, n - 1))))
        d.u_accept.copy_(torch.from_numpy(W.uniforms(rng, (B, n - 1))))
        d.u_final.copy_(torch.from_numpy(W.uniforms(rng, (B,))))
    assert [engine.status_words(t)[0] for t in (b.dstatus, b.vstatus, c.status, l.status)] == [0] * 4


def test_allocation_refuses(torch):
    from speculative_decoding_draft_04_gb300 import _lib, engine
    with pytest.raises(_lib.SpecError):
        engine.DeviceCache.allocate(2, 1, 8, 2, 96, 16, 4, 64, 8, [1.0], [1.0])
    with pytest.raises(_lib.SpecError):
        engine.DeviceCache.allocate(2, 1, 9, 2, 64, 16, 4, 64, 8, [1.0], [1.0])
    with pytest.raises(_lib.SpecError):
        engine.DeviceCache.allocate(2, 2, 8, 2, 64, 16, 4, 64, 8, [1.0], [1.0])
    with pytest.raises(_lib.SpecError):
        engine.DeviceLogprobs.allocate(2, 4, 100, K=33)


def test_example(torch):
    example = runpy.run_path(os.path.join(os.path.dirname(__file__), "..", "examples", "served_cycle.py"))
    out, c = example["serve"](requests=3, cycles=3, prompt=20, V=4000, width=128, layers=2)
    kept = np.arange(20, 23)
    for tokens, lp in out:
        live = (tokens >= 0).cpu().numpy()
        assert (live.sum(1) >= 1).all() and (torch.isfinite(lp).cpu().numpy() == live).all()
        before, kept = kept, kept + live.sum(1)
    assert c.seq_len[c.newest].cpu().tolist() == before.tolist()
