"""The served cycle with requests that have no rows in a step: a pool that runs out, a finished
request, and a new prompt in its slot.  Such a request emits nothing and keeps exactly what it had;
every layer's attention sees the tokens that were kept and no other."""
import os
import runpy

import numpy as np
import pytest

from oracle import serving as S
from tests import serving as H

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE, PAGES = 4, 2, 64, 16, 7
K_SCALE, V_SCALE = 0.00893, 0.00227
NO_PAGES = 256


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.mark.parametrize("side", [False, True])
def test_requests_without_rows(torch, side):
    from speculative_decoding_draft_04_gb300 import engine
    from speculative_decoding_draft_04_gb300 import workloads as W
    w = W.make_workload(W.config("C0"), 3)
    d = engine.DeviceWorkload.from_workload(w)
    b, alone = engine.Buffers.for_workload(d), engine.Buffers.for_workload(d)
    B, n, V = w.B, w.gamma + 1, w.V
    prompts = np.array([30, 20, 12, 5] + [1] * (B - 4), np.int64)[:B]
    rows = int(prompts.sum()) + B * n
    c = engine.DeviceCache.allocate(B, 1, HQ, HKV, D, PAGE, PAGES, 128, rows, [K_SCALE], [V_SCALE])
    l = engine.DeviceLogprobs.allocate(B, n, V, K=2)
    pool = S.Pool(PAGE, range(PAGES), [[] for _ in range(B)], c.block_table.shape[1])
    rng = np.random.default_rng(4)
    stream = torch.cuda.Stream() if side else None
    scales = [np.float64(np.float32(x)) for x in (K_SCALE, V_SCALE)]
    kept = [[np.zeros((0, HKV, D)) for _ in range(B)] for _ in range(2)]

    def attend(base, count):
        """The kept tokens are the first base; append and attend random rows; check them."""
        for which in kept:
            for i in range(B):
                which[i] = which[i][:base[i]]
                assert len(which[i]) == base[i]
        ptr = np.concatenate([[0], np.cumsum(count)])
        T = int(ptr[-1])
        q, k, v = (rng.normal(size=(T, h, D)).astype(np.float32) for h in (HQ, HKV, HKV))
        on = [H.dev(x) for x in (q, k, v)]
        out = torch.zeros((T, HQ, D), dtype=torch.float32, device="cuda")
        torch.cuda.synchronize()
        engine.attend(c, 0, *on, out, stream=stream)
        torch.cuda.synchronize()
        for which, x in enumerate((k, v)):
            code, s = S.store(x.reshape(-1, 16), scales[which])
            x = S.values(code, s, scales[which]).reshape(T, HKV, D)
            for i in range(B):
                kept[which][i] = np.concatenate([kept[which][i], x[ptr[i]:ptr[i + 1]]])
        out = out.double().cpu().numpy()
        for i in range(B):
            see = S.visible(int(count[i]), len(kept[0][i]))
            for h in range(HQ if count[i] else 0):
                kk, vv = (kept[x][i][:, h * HKV // HQ] for x in (0, 1))
                o, _, absv, big = S.attention(q[ptr[i]:ptr[i + 1], h].astype(np.float64), kk, vv, see, D ** -0.5)
                tol = 2.0 ** -22 * np.abs(o) + (2.0 ** -20 + 2.0 ** -17 * big[:, None] + 2.0 ** -15) * absv + 1e-30
                assert (np.abs(out[ptr[i]:ptr[i + 1], h] - o) <= tol).all(), (i, h)

    def room(seq, accept, new):
        base, add, _, _ = pool.step(seq, accept, new, rows)
        return np.array(base), np.array(add)

    def i32(a):
        t = H.dev(np.asarray(a, np.int32))
        torch.cuda.synchronize()
        return t

    seq = np.zeros(B, np.int64)
    seq, count = room(seq, None, prompts)
    engine.make_room(c, i32(prompts))
    attend(seq, count)
    accept = prompts - 1
    on_device = i32(accept)
    state, seen = "filling", []
    for step in range(40):
        new = np.full(B, n)
        if state == "refused":                           # a request leaves, its pages go back
            new[1], state = -1, "finished"
        elif state == "finished":                        # another one takes its place
            prompt = np.where(np.arange(B) == 1, 9, 0)
            seq, count = room(seq, accept, prompt)
            engine.make_room(c, i32(prompt), on_device)
            attend(seq, count)
            assert count[1] == 9
            accept = np.where(np.arange(B) == 1, 8, -1)
            on_device, state = i32(accept), "again"
        seq, count = room(seq, accept, new)
        if state == "filling" and (count == 0).any():
            state = "refused"
        torch.cuda.synchronize()
        engine.served_cycle(d, b, c, l, lambda *a: attend(seq, count), i32(new), on_device, stream)
        torch.cuda.synchronize()
        assert c.seq_len[c.newest].cpu().tolist() == seq.tolist()
        assert c.kv_len.cpu().tolist() == (seq + count).tolist()
        assert c.num_blocks[c.newest].cpu().tolist() == [len(t) for t in pool.tables]
        engine.cycle(d, alone)
        live = count > 0
        accept = np.where(live, alone.accept_len.cpu().numpy(), -1)
        tokens = np.where(live[:, None], alone.out_tokens.cpu().numpy(), -1)
        assert b.accept_len.cpu().tolist() == accept.tolist()
        np.testing.assert_array_equal(b.out_tokens.cpu().numpy(), tokens)
        np.testing.assert_array_equal(np.isnan(l.logprob.cpu().numpy()), tokens < 0)
        assert (l.top_ids.cpu().numpy()[tokens < 0] == -1).all()
        on_device = b.accept_len.clone()
        seen.append((state, live.copy()))
        for u, shape in ((d.u_draft, (B, n - 1)), (d.u_accept, (B, n - 1)), (d.u_final, (B,))):
            u.copy_(torch.from_numpy(W.uniforms(rng, shape)))
        torch.cuda.synchronize()
        if state == "again" and len([1 for s, _ in seen if s == "again"]) == 4:
            break
    refused = next(x for s, x in seen if s == "refused")
    assert not refused.all() and any(x[~refused].any() for s, x in seen if s == "again")
    words = [engine.status_words(t)[0] for t in (b.dstatus, b.vstatus, c.status, l.status)]
    assert words[0] == words[1] == words[3] == 0 and words[2] == NO_PAGES


def test_example_with_a_small_pool(torch):
    example = runpy.run_path(os.path.join(os.path.dirname(__file__), "..", "examples", "served_cycle.py"))
    out, c = example["serve"](requests=3, cycles=8, prompt=20, V=4000, width=128, layers=2, page_size=16, pages=7)
    kept, some = np.arange(20, 23), np.ones(3, bool)
    for tokens, lp in out:
        live = (tokens >= 0).cpu().numpy()
        assert (torch.isfinite(lp).cpu().numpy() == live).all()
        some &= live[:, 0]
        before, kept = kept, kept + live.sum(1)
    assert not some.all() and c.seq_len[c.newest].cpu().tolist() == before.tolist()
