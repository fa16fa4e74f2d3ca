"""Plain float64 oracle of the target model's side of a cycle: block tables and
slot maps, the 4-bit cache, attention over it, and log probabilities.

TEST INFRASTRUCTURE, like spec_oracle.py: only ``tests/`` and the examples'
checks may import or run this module.

One request, one row, one group at a time; definitions, not algorithms:

* ``Pool`` keeps the free pages in a Python list and hands them out in request
  order (the ring of the library is a layout of that list);
* ``store`` rounds a group of 16 numbers to 4 bits: the scale is the 8-bit float
  (1 to 4 exponent bits 0..15, bias 7, 3 mantissa bits, at most 448) nearest
  max|x| / (6 g), the codes the levels nearest x / (scale g), ties to the even
  code; the two quotients and the product scale * g are fp32 numbers, as the
  format defines them;
* ``attention`` is softmax(scale q K^T) V of one request's rows;
* ``logprobs`` is log_softmax, entropy and a sort of one row.
"""
from __future__ import annotations

import math

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALES = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                   for e in range(16) for m in range(8)][:127])


def nearest_even(grid: np.ndarray, x: np.ndarray) -> np.ndarray:
    """Index of the grid value nearest x >= 0 (ascending grid), ties to the even index."""
    x = np.asarray(x, np.float64)
    hi = np.minimum(np.searchsorted(grid, x), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - x, x - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def store(x: np.ndarray, g: float):
    """Codes (0..15) and scale index of groups x [..., 16]; NaN counts as 0."""
    with np.errstate(all="ignore"):
        x = np.where(np.isnan(x), 0, x).astype(np.float32)
        g = np.float32(g)
        t = np.abs(x).max(-1) / (np.float32(6) * g)
        s = nearest_even(SCALES, np.minimum(t, 448))
        r = (SCALES[s].astype(np.float32) * g)[..., None]
        y = np.where(r > 0, x / np.where(r > 0, r, 1), 0).astype(np.float32)
    code = nearest_even(LEVELS, np.minimum(np.abs(y), 6.0)) + 8 * (np.signbit(y) & (r > 0))
    return code.astype(np.uint8), s.astype(np.uint8)


def values(code: np.ndarray, s: np.ndarray, g: float) -> np.ndarray:
    """What codes [..., 16] under scale indexes [...] stand for."""
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * SCALES[s][..., None] * float(np.float32(g))


def block_parts(D: int):
    """Byte ranges of K codes, K scales, V codes, V scales in a block of 16 tokens."""
    return (0, 8 * D), (8 * D, 9 * D), (9 * D, 17 * D), (17 * D, 18 * D)


def write_token(cache: np.ndarray, slot: int, h: int, which: int, x: np.ndarray, g: float) -> np.ndarray:
    """Store one head's key (which 0) or value (1) x [D] at a slot; returns the stored values."""
    D = x.shape[0]
    P = cache.shape[2] * 16
    blk = cache[slot // P, h, slot % P // 16]
    code, s = store(x.reshape(-1, 16), g)
    flat = code.reshape(-1)
    c, sc = block_parts(D)[2 * which:2 * which + 2]
    tok = slot % 16
    blk[c[0] + tok * (D // 2):c[0] + (tok + 1) * (D // 2)] = flat[0::2] | (flat[1::2] << 4)
    blk[sc[0] + tok * (D // 16):sc[0] + (tok + 1) * (D // 16)] = s
    return values(code, s, g).reshape(-1)


def read_tokens(cache: np.ndarray, pages: np.ndarray, h: int, L: int, D: int, which: int, g: float):
    """The first L keys or values of head h over a request's pages, float64 [L, D]."""
    P = cache.shape[2] * 16
    out = np.zeros((L, D))
    (c0, c1), (s0, s1) = block_parts(D)[2 * which:2 * which + 2]
    for at in range(0, L, 16):
        blk = cache[pages[at // P], h, at % P // 16]
        n = min(16, L - at)
        packed = blk[c0:c1].reshape(16, D // 2)[:n]
        code = np.stack([packed & 15, packed >> 4], -1).reshape(n, D // 16, 16)
        out[at:at + n] = values(code, blk[s0:s1].reshape(16, D // 16)[:n], g).reshape(n, D)
    return out


# ------------------------------------------------------------- block tables

class Pool:
    """Requests' pages and the free pages, in plain lists."""

    def __init__(self, page: int, free, tables, stride: int):
        self.page, self.free, self.stride = page, list(free), stride
        self.tables = [list(t) for t in tables]

    def step(self, seq, accept, new, max_rows):
        """One call: (base, appended, slots, positions) with -1-free packed rows."""
        B, P = len(seq), self.page
        base = [0 if new[b] < 0 else seq[b] + (accept[b] if accept is not None else -1) + 1
                for b in range(B)]
        add = [max(0, n) for n in new]

        def missing(b, n):
            return -(-(base[b] + n) // P) - len(self.tables[b])
        pages = rows = 0
        refused = False
        for b in range(B):
            pages += max(0, missing(b, add[b]))
            rows += add[b]
            if add[b] > 0 and (pages > len(self.free) or rows > max_rows):
                refused = True
            if refused:
                add[b] = 0
        taken = [max(0, missing(b, add[b])) for b in range(B)]
        given = [max(0, -missing(b, add[b])) for b in range(B)]
        back, slots, positions = [], [], []
        for b in range(B):
            t = self.tables[b]
            t.extend(self.free.pop(0) for _ in range(taken[b]))
            if given[b]:
                back.extend(t[len(t) - given[b]:])
                del t[len(t) - given[b]:]
            for pos in range(base[b], base[b] + add[b]):
                positions.append(pos)
                slots.append(t[pos // P] * P + pos % P)
        self.free.extend(back)
        return base, add, slots, positions


# ------------------------------------------------------------- attention

def attention(q, k, v, seen, scale):
    """Rows q [n, D] over k, v [L, D] with visibility [n, L]: out, lse, and for error
    bounds sum p |v| and the largest sum |q||k| scale over visible tokens."""
    x = scale * (q @ k.T)
    big = np.where(seen, abs(scale) * (np.abs(q) @ np.abs(k).T), 0).max(-1, initial=0.0)
    x = np.where(seen, x, -math.inf)
    m = x.max(-1, initial=-math.inf)
    e = np.exp(x - np.where(np.isfinite(m), m, 0)[:, None])
    z = e.sum(-1)
    p = e / np.where(z > 0, z, 1)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(z > 0, m + np.log(z), -math.inf)
    return p @ v, lse, p @ np.abs(v), big


def visible(n: int, L: int, bits=None) -> np.ndarray:
    """Rows 0..n-1 of the last n of L tokens: causal, or by their mask words."""
    see = np.zeros((n, L), bool)
    for i in range(n):
        see[i, :L - n] = True
        for t in range(n):
            see[i, L - n + t] = t <= i if bits is None else (
                t // 32 < bits.shape[1] and bool((int(bits[i, t // 32]) >> (t % 32)) & 1))
    return see


# ------------------------------------------------------------- log probabilities

def logprobs(x: np.ndarray, T: float, token: int, K: int):
    """logprob, entropy, ids, log probabilities of one row of logits, and for error
    bounds sum p d^2 (d = distance from the maximum).  None: no distribution."""
    raw = x.astype(np.float64)
    x = raw / T
    m = x.max()
    if not math.isfinite(m) or np.isnan(x).any():
        return None
    d = x - m
    e = np.exp(d)
    z = math.fsum(e)
    lz = math.log(z)
    fin = np.isfinite(d)
    p = e[fin] / z
    H = lz - math.fsum(p * d[fin])
    ids = np.lexsort((np.arange(len(raw)), -raw))[:K]
    return d[token] - lz, H, ids, d[ids] - lz, math.fsum(p * d[fin] ** 2)


# ------------------------------------------------------------- sampling

def sample(x: np.ndarray, T: float, u: float, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """token, logprob, kept of one row of logits, and how near the nearest border is that
    decided them, as a part of the mass.  None: no distribution."""
    raw = x.astype(np.float64)
    if np.isnan(raw).any() or not math.isfinite(raw.max()):
        return None
    order = np.lexsort((np.arange(len(raw)), -raw))
    order = order[np.isfinite(raw[order])]
    if top_k > 0:
        order = order[:top_k]
    w = np.exp((raw - raw.max()) / T)
    near = math.inf
    z = math.fsum(w[order])
    before = np.concatenate([[0.0], np.cumsum(w[order])[:-1]])
    n = len(order)
    if top_p < 1:
        n = min(n, int((before < top_p * z).sum()))
        near = min(near, float(np.abs(before[1:] - top_p * z).min(initial=math.inf)) / z)
    n = min(n, int((w[order] >= min_p).sum()))
    if min_p > 0:
        off = np.abs(w[order] - min_p)
        near = min(near, float(off[off > 0].min(initial=math.inf)) / z)
    kept = np.sort(order[:max(1, n)])
    f = np.cumsum(w[kept])
    z = math.fsum(w[kept])
    at = min(int((f <= u * z).sum()), len(kept) - 1)
    near = min(near, float(np.abs(f - u * z).min()) / z)
    token = int(kept[at])
    return token, (raw[token] - raw.max()) / T - math.log(z), len(kept), near


# ------------------------------------------------------------- norm and rotation

def rotated(x: np.ndarray, rows: np.ndarray, weight=None, eps: float = 1e-6, interleaved: bool = False) -> np.ndarray:
    """fp32 heads x [T, H, D], normed with a weight and their first elements rotated by rows
    [T, R / 2, 2] (cosine, sine); every product and sum rounded to fp32, the norm's factor once."""
    f = np.float32
    with np.errstate(all="ignore"):
        y = x.astype(f)
        if weight is not None:
            mean = (x.astype(np.float64) ** 2).mean(-1, keepdims=True)
            y = (y * (1 / np.sqrt(mean + np.float64(f(eps)))).astype(f)) * weight.astype(f)
        R = 2 * rows.shape[1]
        c, s = rows[:, None, :, 0].astype(f), rows[:, None, :, 1].astype(f)
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if interleaved else (y[..., :R // 2], y[..., R // 2:R])
        out = y.copy()
        p, q = a * c - b * s, b * c + a * s
        if interleaved:
            out[..., 0:R:2], out[..., 1:R:2] = p, q
        else:
            out[..., :R // 2], out[..., R // 2:R] = p, q
    return out
