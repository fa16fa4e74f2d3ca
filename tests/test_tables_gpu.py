"""Block tables and slot maps (spec_block_tables) against the oracle's pool of page lists
(oracle/serving.py).  Whole numbers: everything is equal."""
import numpy as np
import pytest

import serving as H
from oracle import serving as S

pytestmark = pytest.mark.gpu
BAD_LEN, NO_PAGES, BAD_SLOT = 2, 256, 512


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_draft_04_gb300 import build as B
    B.build()
    return t


class State:
    """Host state of B requests over a ring of free pages."""

    def __init__(self, rng, B, page, max_len, spare, head=None, stride_slack=4):
        self.B, self.page = B, page
        self.seq = rng.integers(0, max_len + 1, B)
        self.gamma = 7
        held = -(-(self.seq + self.gamma + 1) // page)
        self.stride = int(held.max()) + stride_slack
        self.pages = int(held.sum()) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((B, self.stride), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :held[b]] = order[at:at + held[b]]
            at += held[b]
        self.held = held
        self.head = int(rng.integers(0, 5 * self.pages)) if head is None else head
        self.ring = np.full(self.pages, -7, np.int32)
        for i, pg in enumerate(order[at:]):
            self.ring[(self.head + i) % self.pages] = pg
        self.tail = self.head + spare

    def pool(self):
        return S.Pool(self.page, [int(self.ring[i % self.pages]) for i in range(self.head, self.tail)],
                      [self.table[b, :self.held[b]].tolist() for b in range(self.B)], self.stride)


def call(torch, s, accept, new, max_rows, repeat=1, stream=None):
    L = H.lib()

    def z(*n, dt=torch.int32):
        return torch.full(n, -99, dtype=dt, device="cuda")
    st = H.new_status()
    t = dict(ring=H.dev(s.ring), table=H.dev(s.table), seq=z(s.B), kv=z(s.B), held=z(s.B),
             pos=z(2, dt=torch.int64), ptr=z(s.B + 1), slots=z(max_rows), positions=z(max_rows))
    for _ in range(repeat):
        L.spec_block_tables(H.dev(s.seq.astype(np.int32)),
                            None if accept is None else H.dev(np.asarray(accept, np.int32)),
                            H.dev(np.asarray(new, np.int32)), H.dev(np.asarray(s.held, np.int32)),
                            H.dev(np.array([s.head, s.tail], np.int64)), t["ring"], t["table"], t["seq"], t["kv"],
                            t["held"], t["pos"], t["ptr"], t["slots"], t["positions"], st, s.page, stream=stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in t.items()}, H.status(st)


def check(s, got, base, add, slots, positions, pool, max_rows):
    np.testing.assert_array_equal(got["seq"], base)
    np.testing.assert_array_equal(got["kv"], np.array(base) + np.array(add))
    np.testing.assert_array_equal(got["ptr"], np.concatenate([[0], np.cumsum(add)]))
    np.testing.assert_array_equal(got["held"], [len(t) for t in pool.tables])
    for b, t in enumerate(pool.tables):
        assert got["table"][b, :len(t)].tolist() == t
    head, tail = got["pos"]
    assert [int(got["ring"][i % s.pages]) for i in range(head, tail)] == pool.free
    pad = [-1] * (max_rows - len(slots))
    assert got["slots"].tolist() == slots + pad
    assert got["positions"].tolist() == positions + pad


@pytest.mark.parametrize("B", [1, 2, 31, 128, 256, 257, 1000, 1025, 4096])
@pytest.mark.parametrize("page", [16, 128])
def test_one_step(torch, B, page):
    rng = np.random.default_rng(B + page)
    s = State(rng, B, page, 300, B + 5)
    accept = rng.integers(-1, 8, B)
    new = rng.integers(-1, 9, B)
    rows = int(np.maximum(new, 0).sum()) + 3
    pool = s.pool()
    want = pool.step(s.seq, accept, new, rows)
    got, st = call(torch, s, accept, new, rows)
    assert st == 0
    check(s, got, *want, pool, rows)


@pytest.mark.parametrize("max_new", [1, 17, 1000])
def test_prompts(torch, max_new):
    rng = np.random.default_rng(max_new)
    B = 50
    s = State(rng, B, 16, 100, B * (max_new // 16 + 2), stride_slack=max_new // 16 + 2)
    new = rng.integers(0, max_new + 1, B)
    rows = int(new.sum())
    pool = s.pool()
    want = pool.step(s.seq, None, new, rows)
    got, st = call(torch, s, None, new, rows)
    assert st == 0
    check(s, got, *want, pool, rows)


@pytest.mark.parametrize("spare", [0, 1, 7, 40])
def test_pool_runs_out(torch, spare):
    rng = np.random.default_rng(spare)
    s = State(rng, 300, 16, 200, spare)
    accept, new = rng.integers(-1, 8, 300), rng.integers(-1, 30, 300)
    rows = int(np.maximum(new, 0).sum())
    pool = s.pool()
    want = pool.step(s.seq, accept, new, rows)
    assert sum(want[1]) < rows
    got, st = call(torch, s, accept, new, rows)
    assert st == NO_PAGES
    check(s, got, *want, pool, rows)


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 100])
def test_rows_run_out(torch, rows):
    rng = np.random.default_rng(rows)
    s = State(rng, 40, 32, 100, 100)
    new = rng.integers(0, 9, 40)
    pool = s.pool()
    want = pool.step(s.seq, None, new, rows)
    got, st = call(torch, s, None, new, rows)
    assert st == NO_PAGES
    check(s, got, *want, pool, rows)


def test_everything_finishes(torch):
    rng = np.random.default_rng(1)
    s = State(rng, 77, 16, 300, 0)
    pool = s.pool()
    want = pool.step(s.seq, None, [-1] * 77, 4)
    got, st = call(torch, s, None, [-1] * 77, 4)
    assert st == 0 and (got["kv"] == 0).all()
    check(s, got, *want, pool, 4)


def test_a_repeated_call_gives_the_same(torch):
    rng = np.random.default_rng(2)
    s = State(rng, 200, 16, 300, 300)
    accept, new = rng.integers(-1, 8, 200), rng.integers(-1, 30, 200)
    rows = int(np.maximum(new, 0).sum())
    a, _ = call(torch, s, accept, new, rows)
    b, _ = call(torch, s, accept, new, rows, repeat=3)
    for k in a:
        np.testing.assert_array_equal(a[k], b[k])


def test_many_steps_lose_no_page(torch):
    """A server's life: state handed from step to step; every page is in one place at each step."""
    rng = np.random.default_rng(3)
    B = 60
    s = State(rng, B, 16, 60, 150, head=0, stride_slack=20)
    for step in range(40):
        accept = rng.integers(-1, 8, B)
        new = rng.integers(0, 9, B)
        new[rng.random(B) < 0.1] = -1
        pool = s.pool()
        # a request keeps no more than it appended
        accept = np.minimum(accept, s.held * s.page - s.seq - 1)
        want = pool.step(s.seq, accept, new, 500)
        got, st = call(torch, s, accept, new, 500)
        check(s, got, *want, pool, 500)
        assert sorted(sum(pool.tables, pool.free)) == list(range(s.pages))
        s.seq, s.held = got["seq"].copy(), got["held"].copy()
        s.table, s.ring = got["table"].copy(), got["ring"].copy()
        s.head, s.tail = (int(x) for x in got["pos"])
        long = s.seq > 200
        s.seq = np.where(long, 0, s.seq)                 # a new request starts with the old one's pages


@pytest.mark.parametrize("field,value", [("seq", -1), ("seq", 10 ** 6), ("held", -1), ("held", 10 ** 6),
                                         ("new", -2), ("new", 2 ** 30), ("accept", -2), ("accept", 2 ** 30)])
def test_a_bad_request_keeps_its_pages_and_the_others_go_on(torch, field, value):
    rng = np.random.default_rng(4)
    B, bad = 9, 4
    s = State(rng, B, 16, 100, 40)
    a = dict(accept=rng.integers(0, 8, B), new=rng.integers(0, 9, B))
    good = s.pool()
    rows = 100
    (s.seq if field == "seq" else s.held if field == "held" else a[field])[bad] = value
    got, st = call(torch, s, a["accept"], a["new"], rows)
    assert st == BAD_LEN
    assert got["kv"][bad] == 0 and got["held"][bad] == s.held[bad] and got["ptr"][bad] == got["ptr"][bad + 1]
    # the others: as if it had asked for nothing
    seq, acc, new = s.seq.copy(), a["accept"].copy(), a["new"].copy()
    mine = len(good.tables[bad]) * 16
    seq[bad], acc[bad], new[bad] = mine, -1, 0
    base, add, slots, positions = good.step(seq, acc, new, rows)
    others = [b for b in range(B) if b != bad]
    np.testing.assert_array_equal(got["kv"][others], (np.array(base) + np.array(add))[others])
    assert got["slots"].tolist() == slots + [-1] * (rows - len(slots))


def test_bad_page_ids_and_a_bad_ring(torch):
    rng = np.random.default_rng(5)
    s = State(rng, 3, 16, 20, 5)
    s.seq[:] = 3
    s.table[1, 0] = s.pages
    got, st = call(torch, s, None, [2, 2, 2], 6)
    assert st == BAD_SLOT and got["slots"][2:4].tolist() == [-1, -1] and (got["slots"][[0, 1, 4, 5]] >= 0).all()
    s = State(rng, 3, 16, 20, 5)
    s.tail = s.head + s.pages + 1
    got, st = call(torch, s, None, [60, 60, 60], 180)
    assert st & BAD_LEN and st & NO_PAGES and got["ptr"][-1] == 0


def test_another_stream(torch):
    rng = np.random.default_rng(6)
    s = State(rng, 20, 16, 100, 30)
    new = rng.integers(0, 9, 20)
    a, _ = call(torch, s, None, new, 200)
    b, _ = call(torch, s, None, new, 200, stream=torch.cuda.Stream())
    for k in a:
        np.testing.assert_array_equal(a[k], b[k])
