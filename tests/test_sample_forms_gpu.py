"""Forms of sampling that the other tests do not reach: every number of CTAs a row, top_k that lists cannot hold,
rows whose mask is a large finite number.  Oracle and tolerances as in test_sample_gpu; a border of min-p is
decided on the logit, against max + T ln(min_p) to 2^-34 of T, so no weight may lie within 2^-33 of min_p, relative
to it, however large the mass is (dense fp32 rows: the oracle's own measure is a part of the mass)."""
import numpy as np
import pytest

from oracle import serving as S
from tests import serving as H
from tests.test_sample_gpu import check, run, torch  # noqa: F401 (torch: a fixture)

pytestmark = pytest.mark.gpu


def check_min_p(torch, x, u, T, min_p, **f):  # noqa: F811
    """check() with min_p of one row of each request: what the mass decides is looked at without min-p's border."""
    tokens, lp, kept, st = run(torch, x, u, T, f.get("top_k"), f.get("top_p"), min_p)
    assert st == 0
    T, min_p = float(np.float32(T)), float(np.float32(min_p))
    p = float(np.float32(f.get("top_p", 1.0)))
    for j in range(x.shape[1]):
        raw, uj = x[0, j].double().cpu().numpy(), float(np.float32(u[j]))
        w = np.exp((raw - raw.max()) / T)
        off = np.abs(w / min_p - 1)
        assert (off[off > 0] > 2.0 ** -33).all(), "the seed has a border next to a decision"
        assert S.sample(raw, T, uj, f.get("top_k", 0), p)[3] > 2.0 ** -32.9
        want, wl, wk, _ = S.sample(raw, T, uj, f.get("top_k", 0), p, min_p)
        order = np.lexsort((np.arange(len(raw)), -raw))[:wk]
        F = np.cumsum(w[np.sort(order)])
        assert np.abs(F / F[-1] - uj).min() > 2.0 ** -32.9
        assert (tokens[0, j], kept[0, j]) == (want, wk), (j, f)
        assert abs(lp[0, j] - wl) <= 2.0 ** -23 * abs(wl) + 2.0 ** -31


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 20, 40, 100, 160, 400])
def test_ctas_a_row(torch, rows, dtype):  # noqa: F811
    """8, 8, 4, 2, 2 and 1 of them with 152 SMs; settings that differ from row to row, eight rows are looked at."""
    rng = np.random.default_rng(rows)
    V = 140000
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    x = (torch.randn((rows, 1, V), generator=gen, device="cuda") * 2 - 5).to(H.storage(torch, dtype))
    u = rng.random(rows).astype(np.float32)
    k, p, m = rng.choice([0, 50, 3000], rows), rng.choice([1.0, 0.5, 0.9], rows), rng.choice([0.0, 0.0, 0.02], rows)
    tokens, lp, kept, st = run(torch, x, u, 0.8, k, p, m)
    assert st == 0
    for b in sorted({0, rows - 1, *rng.integers(0, rows, 6).tolist()}):
        raw = x[b, 0].double().cpu().numpy()
        want, wl, wk, near = S.sample(raw, float(np.float32(0.8)), float(u[b]), int(k[b]), float(np.float32(p[b])),
                                      float(np.float32(m[b])))
        assert near > 2.0 ** -32.9 and (tokens[b, 0], kept[b, 0]) == (want, wk), (b, k[b], p[b], m[b])
        assert abs(lp[b, 0] - wl) <= 2.0 ** -23 * abs(wl) + 2.0 ** -31


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2049, 6000, 50000, 131072])
@pytest.mark.parametrize("mean", [0.0, -10.0])
def test_large_top_k(torch, V, mean, dtype):  # noqa: F811
    """From 2047, about what a list holds, to all entries but one, alone and with the other filters."""
    rng = np.random.default_rng(V)
    x = H.dev(rng.normal(mean, 1.5, (1, 2, V)), H.storage(torch, dtype))
    for k in sorted({2047, 2048, 2049, V // 2, V - 1, V}):
        if 2047 <= k <= V:
            for f in ({}, dict(top_p=0.9), dict(top_p=0.97, min_p=0.001), dict(min_p=0.01)):
                (check_min_p if "min_p" in f else check)(torch, x, rng.random(2), T=0.9, top_k=k, **f)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fill", [-1e9, None])
def test_rows_masked_by_a_finite_number(torch, fill, dtype):  # noqa: F811
    """More entries are left than a list holds; None: the type's lowest value."""
    rng = np.random.default_rng(5)
    V, left = 40000, 6000
    x = H.dev(rng.normal(0.0, 3.0, (1, 2, V)), H.storage(torch, dtype))
    off = np.ones((1, 2, V), bool)
    for j in range(2):
        off[0, j, rng.permutation(V)[:left]] = False
    x.masked_fill_(H.dev(off), torch.finfo(x.dtype).min if fill is None else fill)
    for f in ({}, dict(top_k=20), dict(top_k=2500), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=50, top_p=0.9)):
        check(torch, x, rng.random(2), **f)


def test_the_same_on_every_run(torch):  # noqa: F811
    rng = np.random.default_rng(6)
    x = H.dev(rng.normal(-10.0, 1.0, (30, 1, 50000)), torch.bfloat16)
    u, k = rng.random(30), rng.choice([0, 3000], 30)
    first = run(torch, x, u, 1.0, k, 0.9, None)
    for _ in range(5):
        again = run(torch, x, u, 1.0, k, 0.9, None)
        assert all(np.array_equal(a, b) for a, b in zip(first[:3], again[:3]))
