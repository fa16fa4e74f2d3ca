"""Cases of three more operators of the target model's side of a cycle, with their plain forms.

  sample   a token of each row of logits: temperature, top-k, top-p and min-p, drawn from a given
           uniform number.
  rotary   the rows of a fused projection: queries and keys normed per head and rotated by their
           positions, keys and values rounded to 4 bits and written into the paged cache.
  prefix   attention of a few new tokens of each request over the cache, where groups of requests
           share a long prefix that is held once.

The 4-bit cache is uint8 [num_pages][Hkv][page_size / 16][18 D]: per page and key-value head, blocks
of 16 tokens, each K codes [16][D/2], K scales [16][D/16], V codes [16][D/2], V scales [16][D/16].
A code is a sign, two exponent bits and one mantissa bit (0, 0.5, 1, 1.5, 2, 3, 4, 6), the even
element in the low half of its byte; 16 consecutive elements share one 8-bit scale (four exponent
bits, three mantissa bits).  A key stands for code * scale * k_scale, a value for
code * scale * v_scale.

``run`` computes the plain forms, or calls the library where ``own`` is set.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
# Calibrated scales of a layer's keys and values: about its largest magnitude over 6 * 448.
K_SCALE, V_SCALE = float(np.float32(0.00893)), float(np.float32(0.00227))
EPS = 1e-6


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # First tokens of four requests of the smallest workload, 32-bit logits: latency.
        dict(name="sample-first-b4", op="sample", B=4, n=1, V=1000, dtype="f32", filters="mixed",
             masked=0.0),
        # One plain decoding step of 128 requests, each with its own settings; some follow a grammar
        # that masks most of the vocabulary.
        dict(name="sample-step-b128", op="sample", B=128, n=1, V=32000, dtype="bf16",
             filters="mixed", masked=0.1),
        # The same over a large vocabulary.
        dict(name="sample-step-b256", op="sample", B=256, n=1, V=128256, dtype="bf16",
             filters="mixed", masked=0.1),
        # Sampling at temperatures alone, 32-bit logits of the largest vocabulary.
        dict(name="sample-open-b64", op="sample", B=64, n=1, V=151936, dtype="f32", filters="none",
             masked=0.0),
        # One token of one request in 32-bit storage, small heads: latency.
        dict(name="rotary-one-b1", op="rotary", T=1, Hq=8, Hkv=2, D=64, R=64, page=16, dtype="f32",
             norm=True, interleaved=False, skipped=0.0),
        # The blocks of one verification step of 128 requests.
        dict(name="rotary-block-b128", op="rotary", T=1024, Hq=32, Hkv=8, D=128, R=128, page=64,
             dtype="bf16", norm=True, interleaved=False, skipped=0.05),
        # Prompts: a long run of tokens, an odd number of them.
        dict(name="rotary-prompts", op="rotary", T=30011, Hq=32, Hkv=8, D=128, R=128, page=64,
             dtype="bf16", norm=True, interleaved=False, skipped=0.0),
        # Large heads of which a quarter is rotated, pairs side by side, no norm, 32-bit storage.
        dict(name="rotary-partial-f32", op="rotary", T=4099, Hq=16, Hkv=4, D=256, R=64, page=32,
             dtype="f32", norm=False, interleaved=True, skipped=0.0),
        # One token of four requests behind an instruction of 2000 tokens: latency.
        dict(name="prefix-one-b4", op="prefix", groups="4", prefixes="2000", Hq=16, Hkv=4, D=64,
             page=32, dtype="bf16", kind="one", max_new=1, min_own=1, max_own=100),
        # Plain decoding of 64 requests about one document.
        dict(name="prefix-one-b64", op="prefix", groups="64", prefixes="16384", Hq=32, Hkv=8, D=128,
             page=64, dtype="bf16", kind="one", max_new=1, min_own=64, max_own=2048),
        # A verification step of 128 requests of three services, some without a prefix.
        dict(name="prefix-block-b128", op="prefix", groups="70 1 41 16",
             prefixes="8192 0 4100 777", Hq=32, Hkv=8, D=128, page=64, dtype="bf16", kind="block",
             max_new=8, min_own=8, max_own=1024),
        # Trees of 24 candidate slots and the anchor behind a long prefix.
        dict(name="prefix-tree-b32", op="prefix", groups="32", prefixes="32768", Hq=32, Hkv=8, D=128,
             page=32, dtype="bf16", kind="tree", max_new=25, min_own=25, max_own=512),
    ]


def _numbers(text):
    return [int(x) for x in text.split()]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "rotary", "prefix"])
    if op == "sample":
        V = _log_int(rng, 16, 151936)
        rows = _log_int(rng, 1, max(2, min(1024, 64 * 151936 // V)))
        n = min(rows, rng.choice([1, 1, 1, rng.randint(2, 8)]))
        return dict(op=op, B=max(1, rows // n), n=n, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    filters=rng.choice(["mixed", "mixed", "top_k", "top_p", "min_p", "none"]),
                    masked=rng.choice([0.0, 0.1, 0.5]))
    if op == "rotary":
        D = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([h for h in (1, 2, 3, 4, 8) if h * D <= 1024])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 7])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 30011 * 48 * 128 * 2 // ((Hq + 2 * Hkv) * D * SIZES[dtype])
        return dict(op=op, T=_log_int(rng, 1, min(30011, most)), Hq=Hq, Hkv=Hkv, D=D,
                    R=rng.choice([D, D, D // 2, 32]), page=rng.choice([16, 32, 64, 128]), dtype=dtype,
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.4,
                    skipped=rng.choice([0.0, 0.1]))
    kind = rng.choice(["one", "one", "block", "tree"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([h for h in (1, 2, 4, 8) if h * D <= 1024])
    group = rng.choice([1, 2, 3, 4, 6, 8])
    max_new = 1 if kind == "one" else rng.randint(2, 9) if kind == "block" else rng.randint(4, 33)
    B = _log_int(rng, 1, max(1, min(128, 1200 // max_new)))
    parts = min(B, rng.choice([1, 1, 2, 3, 5]))
    cuts = sorted(rng.sample(range(1, B), parts - 1)) if parts > 1 else []
    groups = [b - a for a, b in zip([0] + cuts, cuts + [B])]
    # rows x tokens x heads x elements stay below the largest listed case, 32-bit storage costs more
    dtype = rng.choice(["bf16", "bf16", "f32"])
    room = 32 * 25 * 32768 * 32 * 128 // (B * max_new * Hkv * group * D)
    if dtype == "f32" or D == 256:
        room //= 8
    prefixes = [rng.choice([0, 1]) * _log_int(rng, 1, max(2, min(32768, room))) if parts > 1
                else _log_int(rng, 1, max(2, min(32768, room))) for _ in groups]
    max_own = max(max_new + 1, _log_int(rng, 1, max(2, min(2048, room))))
    return dict(op=op, groups=" ".join(map(str, groups)), prefixes=" ".join(map(str, prefixes)),
                Hq=Hkv * group, Hkv=Hkv, D=D,
                page=rng.choice([16, 32, 64, 128]), dtype=dtype, kind=kind, max_new=max_new,
                min_own=max_new, max_own=max_own)


# ------------------------------------------------------------------ the inputs

def _host_rng(case, seed):
    return np.random.default_rng([seed & 0x7FFFFFFF] + [ord(ch) for ch in case["op"]])


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(DEV)


def _status():
    return torch.zeros(4, dtype=torch.int32, device=DEV)


def _parts(cache, D):
    """Views of a cache's K codes, K scales, V codes, V scales: [pages, P/16, 16, H, ...]."""
    c = cache.permute(0, 2, 1, 3)
    return (c[..., :8 * D].unflatten(-1, (16, D // 2)).transpose(2, 3),
            c[..., 8 * D:9 * D].unflatten(-1, (16, D // 16)).transpose(2, 3),
            c[..., 9 * D:17 * D].unflatten(-1, (16, D // 2)).transpose(2, 3),
            c[..., 17 * D:].unflatten(-1, (16, D // 16)).transpose(2, 3))


def _scalar(v):
    # A number in 32 bits on the GPU: division by a tensor is division, by a host number it is not.
    return torch.full((), v, dtype=torch.float32, device=DEV)


def _to_4bit(x, g):
    """Codes (packed), scale bytes and the values they stand for of x [..., D] in 32 bits."""
    xg = x.unflatten(-1, (-1, 16))
    amax = xg.abs().amax(-1)
    s8 = (amax / _scalar(6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    r = (s8.float() * _scalar(g)).unsqueeze(-1)
    y = torch.where(r > 0, xg / r, torch.zeros((), device=x.device))
    m = y.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75).to(torch.uint8) + (m > 1.25).to(torch.uint8)
            + (m >= 1.75).to(torch.uint8) + (m > 2.5).to(torch.uint8) + (m >= 3.5).to(torch.uint8)
            + (m > 5.0).to(torch.uint8))
    value = torch.tensor(LEVELS, device=x.device).index_select(0, code.int().flatten()).view_as(y)
    value = torch.where(torch.signbit(y), -value, value) * s8.float().unsqueeze(-1) * _scalar(g)
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.view(torch.uint8), value.flatten(-2)


def _from_4bit(codes, scales, g):
    """32-bit values of packed codes [..., D/2] and scale bytes [..., D/16]."""
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    x = table.index_select(0, c.int().flatten()).view(c.shape).unflatten(-1, (-1, 16))
    s = scales.contiguous().view(torch.float8_e4m3fn).float() * _scalar(g)
    return (x * s.unsqueeze(-1)).flatten(-2)


def _random_cache(gen, pages, H, page, D):
    """A cache of random keys (channels of different size) and values."""
    cache = torch.empty((pages, H, page // 16, 18 * D), dtype=torch.uint8, device=DEV)
    kc, ks, vc, vs = _parts(cache, D)
    channel = torch.exp(0.5 * torch.randn((H, D), generator=gen, device=DEV))
    step = max(1, (1 << 26) // (H * page * D))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        k = torch.randn((n, page // 16, 16, H, D), generator=gen, device=DEV) * channel
        v = torch.randn((n, page // 16, 16, H, D), generator=gen, device=DEV)
        kc[at:at + n], ks[at:at + n], _ = _to_4bit(k, K_SCALE)
        vc[at:at + n], vs[at:at + n], _ = _to_4bit(v, V_SCALE)
    return cache


def _prepare_sample(case, rng, gen):
    B, n, V = case["B"], case["n"], case["V"]
    # Frequent and rare tokens (a power law) under noise of another size from request to request:
    # flat rows whose nucleus has thousands of tokens, and peaked ones.
    spread = _dev(rng.uniform(1.5, 4.0, (B, 1, 1)), np.float32)
    logits = torch.empty((B, n, V), dtype=DTYPES[case["dtype"]], device=DEV)
    for b in range(0, B, 64):
        part = logits[b:b + 64]
        rare = torch.log1p(V * torch.rand(part.shape, generator=gen, device=DEV))
        x = spread[b:b + 64] * torch.randn(part.shape, generator=gen, device=DEV) - 1.1 * rare
        part.copy_(x)
    for b in np.flatnonzero(rng.random(B) < case["masked"]):         # a grammar's few tokens
        off = torch.rand((n, V), generator=gen, device=DEV) < 0.95
        off[:, int(rng.integers(0, V))] = False
        logits[int(b)].masked_fill_(off, -math.inf)
    kinds = dict(mixed=("none", "top_k", "top_p", "min_p", "both", "all"), none=("none",),
                 top_k=("top_k",), top_p=("top_p",), min_p=("min_p",))[case["filters"]]
    kind = rng.choice(kinds, B)
    k = np.where(np.isin(kind, ("top_k", "both", "all")), rng.choice([1, 8, 20, 50, 200, 1000], B), 0)
    p = np.where(np.isin(kind, ("top_p", "both", "all")), rng.choice([0.8, 0.9, 0.95], B), 1.0)
    m = np.where(np.isin(kind, ("min_p", "all")), rng.choice([0.01, 0.05, 0.1], B), 0.0)
    plain = case["filters"] == "none"
    return dict(logits=logits, u=torch.rand((B, n), generator=gen, device=DEV),
                temperature=_dev(rng.choice([0.6, 0.7, 1.0], B), np.float32),
                top_k=None if plain else _dev(k, np.int32), top_p=None if plain else _dev(p, np.float32),
                min_p=None if plain else _dev(m, np.float32),
                tokens=torch.empty((B, n), dtype=torch.int32, device=DEV),
                logprob=torch.empty((B, n), dtype=torch.float32, device=DEV),
                kept=torch.empty((B, n), dtype=torch.int32, device=DEV), status=_status())


def _rope(length, R):
    """cos and sin of position * 10000^(-2 i / R): [length][R / 2][2], angles in 64 bits."""
    f = 10000.0 ** (-2.0 * torch.arange(R // 2, dtype=torch.float64, device=DEV) / R)
    a = torch.arange(length, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.stack([torch.cos(a), torch.sin(a)], -1).float()


def _prepare_rotary(case, rng, gen):
    T, Hq, H, D, P = case["T"], case["Hq"], case["Hkv"], case["D"], case["page"]
    dt = DTYPES[case["dtype"]]
    qkv = torch.empty((T, Hq + 2 * H, D), dtype=dt, device=DEV)      # a fused projection's rows
    qkv.copy_(torch.randn(qkv.shape, generator=gen, device=DEV))
    channel = torch.exp(0.5 * torch.randn((H, D), generator=gen, device=DEV))
    qkv[:, Hq:Hq + H].mul_(channel.to(dt))
    length = 32768
    if T <= 4096:                                    # blocks of up to eight tokens of many requests
        slots = rng.permutation((-(-T // P) + 3) * P)[:T]
        positions = np.minimum(rng.integers(0, length, -(-T // 8)).repeat(8)[:T] + np.arange(T) % 8, length - 1)
    else:                                            # prompts: whole pages in random order
        at = np.arange(T)
        slots = rng.permutation(-(-T // P) + 3)[at // P] * P + at % P
        positions = at % 8192
    slots[rng.random(T) < case["skipped"]] = -1
    pages = -(-T // P) + 3

    def weight():
        w = 1.0 + 0.2 * torch.randn(D, generator=gen, device=DEV)
        return w.to(dt) if case["norm"] else None
    return dict(D=D, R=case["R"], page=P, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H], v=qkv[:, Hq + H:],
                interleaved=case["interleaved"], q_weight=weight(), k_weight=weight(),
                positions=_dev(positions, np.int32), slots=_dev(slots, np.int32),
                rope=_rope(length, case["R"]),
                cache=torch.zeros((pages, H, P // 16, 18 * D), dtype=torch.uint8, device=DEV),
                q_out=torch.zeros((T, Hq, D), dtype=dt, device=DEV),
                k_stored=torch.empty((T, H, D), dtype=dt, device=DEV),
                v_stored=torch.empty((T, H, D), dtype=dt, device=DEV), status=_status())


def _prepare_prefix(case, rng, gen):
    P, D, Hkv, Hq = case["page"], case["D"], case["Hkv"], case["Hq"]
    groups, prefixes = np.array(_numbers(case["groups"])), np.array(_numbers(case["prefixes"]))
    B, new = int(groups.sum()), case["max_new"]
    n = rng.permutation(2 + np.arange(B) % max(1, new - 1)) if case["kind"] == "block" else np.full(B, new)
    kv = np.maximum(n, rng.integers(case["min_own"], case["max_own"] + 1, B))
    blocks, held = -(-kv // P), -(-prefixes // P)
    pages = int(blocks.sum() + held.sum()) + 5
    perm = rng.permutation(pages)

    def table(count, wide, ids):
        t = np.full((len(count), max(1, wide)), -1, np.int32)
        t[np.arange(t.shape[1])[None, :] < count[:, None]] = ids
        return _dev(t, np.int32)
    own_table = table(blocks, -(-case["max_own"] // P), perm[:blocks.sum()])
    prefix_table = table(held, int(held.max()), perm[blocks.sum():blocks.sum() + held.sum()])
    ptr = np.concatenate([[0], np.cumsum(n)])
    T = int(ptr[-1])
    mask = None
    if case["kind"] == "tree":                       # row i of a request sees itself and its ancestors
        words = -(-new // 32)
        bits = np.zeros((B, new, words), np.uint32)
        for i in range(new):
            if i:
                bits[:, i] = bits[np.arange(B), rng.integers(max(0, i - 6), i, B)]
            bits[:, i, i // 32] |= np.uint32(1 << (i % 32))
        mask = torch.from_numpy(bits.reshape(T, words).view(np.int32)).to(DEV)
    dt = DTYPES[case["dtype"]]
    cuts = np.concatenate([[0], np.cumsum(groups)])
    return dict(page=P, D=D, Hq=Hq, Hkv=Hkv, B=B, max_new=int(n.max()), max_own=int(kv.max()), mask=mask,
                rows=ptr[cuts].tolist(), lengths=prefixes.tolist(), softmax_scale=1.0 / math.sqrt(D),
                q=torch.randn((T, Hq, D), generator=gen, device=DEV).to(dt),
                cache=_random_cache(gen, pages, Hkv, P, D), block_table=own_table, kv_len=_dev(kv, np.int32),
                row_ptr=_dev(ptr, np.int32), prefix_table=prefix_table, prefix_len=_dev(prefixes, np.int32),
                group_ptr=_dev(cuts, np.int32), out=torch.empty((T, Hq, D), dtype=dt, device=DEV),
                lse=torch.empty((T, Hq), dtype=torch.float32, device=DEV), status=_status())


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    make = dict(sample=_prepare_sample, rotary=_prepare_rotary, prefix=_prepare_prefix)[case["op"]]
    return dict(make(case, _host_rng(case, seed), gen), op=case["op"])


# ------------------------------------------------------------- the plain forms

def _plain_sample(s):
    # sums in 64 bits: a uniform number lies next to one of a large vocabulary's borders
    x = s["logits"]
    V = x.shape[-1]
    d = x.double()
    d = (d - d.amax(-1, keepdim=True)) / s["temperature"].double()[:, None, None]
    w = torch.exp(d)
    keep = torch.isfinite(x)
    if s["top_k"] is not None:
        order = torch.sort(x, dim=-1, descending=True, stable=True).indices
        place = torch.arange(V, device=x.device)
        k = s["top_k"][:, None, None]
        among = (place < torch.where(k > 0, k, V)) & keep.gather(-1, order)
        mass = torch.where(among, w.gather(-1, order), 0.0)
        total = mass.cumsum(-1)
        before = torch.cat([torch.zeros_like(total[..., :1]), total[..., :-1]], -1)
        p = s["top_p"].double()[:, None, None]
        among &= (before < p * total[..., -1:]) | (p >= 1) | (place == 0)
        among &= (mass >= s["min_p"].double()[:, None, None]) | (place == 0)
        keep = torch.zeros_like(among).scatter_(-1, order, among)
    f = torch.where(keep, w, 0.0).cumsum(-1)
    z = f[..., -1]
    at = (f <= (s["u"].double() * z).unsqueeze(-1)).sum(-1)
    last = torch.where(keep, torch.arange(V, device=x.device), 0).amax(-1)
    token = torch.minimum(at, last)
    logprob = d.gather(-1, token.unsqueeze(-1)).squeeze(-1) - torch.log(z)
    return dict(tokens=token.int(), logprob=logprob.float(), kept=keep.sum(-1).int())


def _rotate(x, rows, R, interleaved):
    """x [T, H, D] with its first R elements rotated by rows [T, R / 2, 2]."""
    c, s = rows[:, None, :, 0], rows[:, None, :, 1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    y = (a * c - b * s, b * c + a * s)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., R:]], -1)


def _plain_rotary(s):
    P, D = s["page"], s["D"]
    rows = s["rope"][s["positions"].long()]

    def turned(x, weight):
        y = x.float()
        if weight is not None:
            # the mean in 64 bits: what the cache holds turns on the last bit next to a border
            mean = x.double().square().mean(-1, keepdim=True)
            y = y * torch.rsqrt(mean + EPS).float() * weight.float()
        return _rotate(y, rows, s["R"], s["interleaved"]).to(x.dtype)
    live = s["slots"] >= 0
    keep = live[:, None, None]
    q_out = torch.where(keep, turned(s["q"], s["q_weight"]), s["q_out"])
    kc, ks, vc, vs = _parts(s["cache"], D)
    slot = s["slots"][live].long()
    at = (slot // P, slot % P // 16, slot % 16)
    codes, scales, k_val = _to_4bit(turned(s["k"], s["k_weight"]).float(), K_SCALE)
    kc[at], ks[at] = codes[live], scales[live]
    codes, scales, v_val = _to_4bit(s["v"].float(), V_SCALE)
    vc[at], vs[at] = codes[live], scales[live]
    zero = torch.zeros((), device=DEV)
    return dict(q_out=q_out, k_stored=torch.where(keep, k_val, zero).to(s["k"].dtype),
                v_stored=torch.where(keep, v_val, zero).to(s["v"].dtype))


def _tokens_of(cache, table, length, P, D):
    """32-bit keys and values [..., length, Hkv, D] of the tables' first tokens."""
    pos = torch.arange(length, device=DEV)
    page = table[..., pos // P].clamp(min=0)
    at = (page, (pos % P // 16).expand(page.shape), (pos % 16).expand(page.shape))
    kc, ks, vc, vs = _parts(cache, D)
    return _from_4bit(kc[at], ks[at], K_SCALE), _from_4bit(vc[at], vs[at], V_SCALE)


def _part_of(x, v):
    """Maximum, sum and weighted values of scores x [..., rows, tokens]; maximum -inf of none."""
    if x.shape[-1] == 0:
        none = x.new_full(x.shape[:-1] + (1,), -math.inf)
        return none, torch.zeros_like(none), x.new_zeros(x.shape[:-1] + (v.shape[-1],))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    return m, e.sum(-1, keepdim=True), torch.matmul(e, v)


def _plain_prefix(s):
    P, D, B, Hkv, n, L = s["page"], s["D"], s["B"], s["Hkv"], s["max_new"], s["max_own"]
    G = s["Hq"] // Hkv
    T = s["q"].shape[0]
    # ---- the requests' own tokens
    k, v = _tokens_of(s["cache"], s["block_table"], L, P, D)
    pos, row = torch.arange(L, device=DEV), torch.arange(n, device=DEV)
    there = pos < s["kv_len"][:, None]
    ptr = s["row_ptr"]
    fresh = ptr[1:] - ptr[:-1]
    rows = (ptr[:-1, None] + row).clamp(max=T - 1)
    q = s["q"][rows].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["softmax_scale"]
    ctx = (s["kv_len"] - fresh)[:, None, None]
    if s["mask"] is None:
        seen = pos <= ctx + row[:, None]
    else:
        tail = (pos - ctx).expand(B, n, L)
        word = s["mask"][rows].gather(-1, (tail.clamp(0, 32 * s["mask"].shape[1] - 1) // 32))
        seen = (tail < 0) | ((word >> (tail.clamp(min=0) % 32)) & 1).bool()
    seen = (seen & there[:, None]).repeat(1, G, 1)[:, None]
    v = torch.where(there[..., None, None], v, 0.0).permute(0, 2, 1, 3)
    live = row < fresh[:, None]
    own_part = [t.view(B, Hkv, G, n, -1).permute(0, 3, 1, 2, 4)[live]
                for t in _part_of(torch.where(seen, x, -math.inf), v)]
    # ---- the prefix of each group, once for all its rows
    shared = [torch.empty_like(t) for t in own_part]
    for g, length in enumerate(s["lengths"]):
        r0, r1 = s["rows"][g], s["rows"][g + 1]
        k, v = _tokens_of(s["cache"], s["prefix_table"][g], length, P, D)
        q = s["q"][r0:r1].float().view(r1 - r0, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        x = torch.matmul(q, k.permute(1, 2, 0)) * s["softmax_scale"]
        for t, y in zip(shared, _part_of(x, v.transpose(0, 1))):
            t[r0:r1] = y.view(Hkv, r1 - r0, G, -1).transpose(0, 1)
    m = torch.maximum(own_part[0], shared[0])
    ref = torch.where(torch.isfinite(m), m, 0.0)
    a, b = torch.exp(own_part[0] - ref), torch.exp(shared[0] - ref)
    total = a * own_part[1] + b * shared[1]
    y = (a * own_part[2] + b * shared[2]) / torch.where(total > 0, total, 1.0)
    return dict(out=y.view(T, s["Hq"], D).to(s["q"].dtype), lse=(m + torch.log(total)).view(T, s["Hq"]))


# -------------------------------------------------------------- the operators

def _own_sample(s):
    from speculative_decoding_draft_04_gb300 import _lib
    _lib.spec_sample(s["logits"], s["u"], s["tokens"], s["status"], temperature=s["temperature"],
                     top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], logprob=s["logprob"],
                     kept=s["kept"])
    return dict(tokens=s["tokens"], logprob=s["logprob"], kept=s["kept"])


def _own_rotary(s):
    from speculative_decoding_draft_04_gb300 import _lib
    _lib.spec_rotary_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"], s["q_out"],
                            s["cache"], s["status"], K_SCALE, V_SCALE, q_weight=s["q_weight"],
                            k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"],
                            k_stored=s["k_stored"], v_stored=s["v_stored"])
    return dict(q_out=s["q_out"], k_stored=s["k_stored"], v_stored=s["v_stored"])


def _own_prefix(s):
    from speculative_decoding_draft_04_gb300 import _lib
    if "workspace" not in s:
        size = _lib.spec_prefix_attention_workspace_bytes(s["q"].shape[0], s["Hq"], s["Hkv"], s["D"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    _lib.spec_prefix_attention(s["q"], s["cache"], s["block_table"], s["kv_len"], s["row_ptr"],
                               s["prefix_table"], s["prefix_len"], s["group_ptr"], s["out"], s["status"],
                               s["workspace"], s["softmax_scale"], K_SCALE, V_SCALE, tree_mask=s["mask"],
                               lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def run(state):
    if own:
        return dict(sample=_own_sample, rotary=_own_rotary, prefix=_own_prefix)[state["op"]](state)
    return dict(sample=_plain_sample, rotary=_plain_rotary, prefix=_plain_prefix)[state["op"]](state)


# ------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "sample":
        rows = case["B"] * case["n"]
        return dict(bytes=rows * (case["V"] * SIZES[case["dtype"]] + 16) + 16 * case["B"],
                    flops=6 * rows * case["V"])
    if op == "rotary":
        # the projection's rows in, queries, cache and the values as stored out, a row of the table
        # of rotations for each token
        T, D, s = case["T"], case["D"], SIZES[case["dtype"]]
        q, kv = T * case["Hq"] * D, 2 * T * case["Hkv"] * D
        return dict(bytes=2 * s * (q + kv) + kv * 9 / 16 + T * (4 * case["R"] + 8), flops=6 * q + 8 * kv)
    groups, prefixes, D = _numbers(case["groups"]), _numbers(case["prefixes"]), case["D"]
    B = sum(groups)
    new = case["max_new"] if case["kind"] != "block" else (min(2, case["max_new"]) + case["max_new"]) / 2
    own_tokens = (case["min_own"] + case["max_own"]) / 2
    tokens = sum(prefixes) + B * own_tokens
    rows = B * new * case["Hq"]
    seen = sum(g * (p + own_tokens) for g, p in zip(groups, prefixes))
    return dict(bytes=tokens * case["Hkv"] * D * 9 / 8 + rows * D * 2 * SIZES[case["dtype"]],
                flops=4 * seen * new * case["Hq"] * D)


# ----------------------------------------------------------------- in 64 bits

def _exact_sample(s):
    B, n, V = s["logits"].shape
    logprob = torch.empty((B, n), dtype=torch.float64, device=DEV)
    for b in range(B):
        for j in range(n):
            x = s["logits"][b, j].double() / s["temperature"][b].double()
            # the distribution over the ranks, which equal entries share in any order
            y, ids = torch.sort(x, descending=True, stable=True)
            count = int((y > -math.inf).sum())
            if s["top_k"] is not None:
                k = int(s["top_k"][b])
                count = min(count, k) if k > 0 else count
                prob = torch.softmax(y[:count], -1)
                p, floor = s["top_p"][b].double(), s["min_p"][b].double()
                if p < 1:
                    count = max(1, min(count, int((prob.cumsum(-1) - prob < p).sum())))
                count = max(1, min(count, int((prob >= floor * prob[0]).sum())))
            ids = ids[:count].sort().values
            logp = torch.log_softmax(x[ids], -1)
            at = torch.searchsorted(torch.exp(logp).cumsum(-1), s["u"][b, j].double(), right=True)
            logprob[b, j] = logp[at.clamp(max=count - 1)]
    return dict(tokens=None, logprob=logprob, kept=None)


def _exact_levels(y):
    """The nearest 4-bit level of |y| in 64 bits, ties to the even code."""
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=y.device)
    hi = torch.searchsorted(levels, y.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    up, down = levels[hi] - y, y - levels[lo]
    return levels[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]


def _exact_rotary(s):
    R, live = s["R"], s["slots"] >= 0
    q = s["q"].double()
    if s["q_weight"] is not None:
        q = q / torch.sqrt((q * q).mean(-1, keepdim=True) + EPS) * s["q_weight"].double()
    pairs = q[..., :R].unflatten(-1, (R // 2, 2) if s["interleaved"] else (2, R // 2))
    if not s["interleaved"]:
        pairs = pairs.transpose(-1, -2)
    turn = torch.view_as_complex(s["rope"].double())[s["positions"].long()][:, None]
    pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    if not s["interleaved"]:
        pairs = pairs.transpose(-1, -2)
    q = torch.cat([pairs.flatten(-2), q[..., R:]], -1)
    q[~live] = s["q_out"][~live].double()
    # values: the scale and the code nearest in 64 bits
    z = s["v"].double().unflatten(-1, (-1, 16))
    t = (z.abs().amax(-1) / (6.0 * V_SCALE)).clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
    r = (torch.round(t / step) * step * V_SCALE).unsqueeze(-1)
    v = (torch.sign(z) * _exact_levels((z.abs() / torch.where(r > 0, r, 1.0)).clamp(max=6.0)) * r).flatten(-2)
    v[~live] = 0.0
    # keys are rounded to their type before the 4 bits: what is held has no value in 64 bits
    return dict(q_out=q, k_stored=None, v_stored=v)


def _exact_prefix(s):
    D, P, Hkv = s["D"], s["page"], s["Hkv"]
    G = s["Hq"] // Hkv
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)

    def value(codes, scales, g):
        c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
        x = torch.where(c >= 8, -1.0, 1.0).double() * levels[c % 8]
        e, f = scales.long() // 8 % 16, (scales.long() % 8).double()
        sc = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2(e.double() - 7))
        return x * sc.repeat_interleave(16, -1) * g

    def tokens(table, length, h):
        block = s["cache"][table[:-(-length // P)].long(), h].flatten(0, 1)
        k = value(block[:, :8 * D].reshape(-1, D // 2), block[:, 8 * D:9 * D].reshape(-1, D // 16), K_SCALE)
        v = value(block[:, 9 * D:17 * D].reshape(-1, D // 2), block[:, 17 * D:].reshape(-1, D // 16), V_SCALE)
        return k[:length], v[:length]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    ptr, kv, cuts = s["row_ptr"].tolist(), s["kv_len"].tolist(), s["group_ptr"].tolist()
    for h in range(Hkv):
        for g, length in enumerate(s["lengths"]):
            pk, pv = tokens(s["prefix_table"][g], length, h)
            for b in range(cuts[g], cuts[g + 1]):
                n, L = ptr[b + 1] - ptr[b], kv[b]
                ok, ov = tokens(s["block_table"][b], L, h)
                see = torch.ones((n, length + L), dtype=torch.bool, device=DEV)
                if s["mask"] is None:
                    see = torch.tril(see, diagonal=length + L - n)
                else:
                    words = s["mask"][ptr[b]:ptr[b + 1]].long() & 0xFFFFFFFF
                    bits = (words[:, :, None] >> torch.arange(32, device=DEV)) & 1
                    see[:, length + L - n:] = bits.flatten(1)[:, :n].bool()
                q = s["q"][ptr[b]:ptr[b + 1], h * G:(h + 1) * G].double().reshape(n * G, D)
                x = torch.cat([q @ pk.T, q @ ok.T], 1).view(n, G, length + L) * s["softmax_scale"]
                x = x.masked_fill(~see[:, None], -math.inf)
                top = torch.logsumexp(x, -1)
                prob = torch.exp(x - top.unsqueeze(-1)).view(n * G, -1)
                lse[ptr[b]:ptr[b + 1], h * G:(h + 1) * G] = top
                out[ptr[b]:ptr[b + 1], h * G:(h + 1) * G] = (prob[:, :length] @ pv + prob[:, length:] @ ov).view(n, G, D)
    return dict(out=out, lse=lse)


def exact(case, seed):
    return dict(sample=_exact_sample, rotary=_exact_rotary, prefix=_exact_prefix)[case["op"]](prepare(case, seed))
