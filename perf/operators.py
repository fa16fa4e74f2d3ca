"""Cases of the serving operators around one speculative cycle, with their plain forms.

Four operators of the target model's side of a cycle:

  tables     block tables and slot maps from request lengths: requests keep the tokens that
             verification accepted, ask for room for the next block, pages move between a ring of
             free pages and the requests' block tables, and every new token gets its slot.
  append     new keys and values rounded to 4 bits and written into the paged cache at their slots.
  attention  attention of a few new tokens of each request (one, a drafted block, or a tree with
             its ancestor mask) over that cache.
  logprobs   log probability of given tokens, entropy, and the top alternatives of target logits.

The 4-bit cache is uint8 [num_pages][Hkv][page_size / 16][18 D]: per page and key-value head, blocks
of 16 tokens, each K codes [16][D/2], K scales [16][D/16], V codes [16][D/2], V scales [16][D/16].
A code is a sign, two exponent bits and one mantissa bit (0, 0.5, 1, 1.5, 2, 3, 4, 6), the even
element in the low half of its byte; 16 consecutive elements share one 8-bit scale (four exponent
bits, three mantissa bits).  A key stands for code * scale * k_scale, a value for
code * scale * v_scale.

``run`` computes the plain forms in 32 bits, or calls the library where ``own`` is set.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
# Calibrated scales of a layer's keys and values: about its largest magnitude over 6 * 448.
K_SCALE, V_SCALE = float(np.float32(0.00893)), float(np.float32(0.00227))


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # One step of a verification server: 128 requests, each keeping its accepted tokens and
        # asking for its next block of up to seven drafted tokens and the anchor.
        dict(name="tables-block-b128", op="tables", B=128, page=64, max_len=8192, max_new=8,
             finished=0.05),
        # Admission of a large batch: prompts of up to 1024 tokens enter in small pages.
        dict(name="tables-prompts-b2048", op="tables", B=2048, page=16, max_len=256, max_new=1024,
             finished=0.1),
        # The block of one step of 128 requests: keys and values are slices of a fused projection.
        dict(name="append-block-b128", op="append", T=1024, H=8, D=128, page=64, dtype="bf16",
             fused=True, skipped=0.05),
        # Prompts: a long run of tokens, an odd number of them.
        dict(name="append-prompts", op="append", T=65553, H=8, D=128, page=64, dtype="bf16",
             fused=False, skipped=0.0),
        # One token of one request in 32-bit storage, small heads, small pages: latency.
        dict(name="attention-one-b1", op="attention", B=1, Hq=8, Hkv=2, D=64, page=16, dtype="f32",
             kind="one", max_new=1, min_len=777, max_len=777),
        # Plain decoding next to speculation: one token of each of 32 requests.
        dict(name="attention-one-b32", op="attention", B=32, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16", kind="one", max_new=1, min_len=200, max_len=16384),
        # The verification pass of 128 requests with ragged verify lengths 1..7 (and the anchor).
        dict(name="attention-block-b128", op="attention", B=128, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16", kind="block", max_new=8, min_len=64, max_len=8192),
        # A tree of 24 candidate slots and the anchor, ancestors visible only.
        dict(name="attention-tree-b32", op="attention", B=32, Hq=32, Hkv=8, D=128, page=32,
             dtype="bf16", kind="tree", max_new=25, min_len=25, max_len=4096),
        # Few requests with long contexts: the long axis has to be split.
        dict(name="attention-block-long-b4", op="attention", B=4, Hq=32, Hkv=8, D=128, page=128,
             dtype="bf16", kind="block", max_new=8, min_len=50000, max_len=131072),
        # Four requests of the smallest workload, 32-bit logits.
        dict(name="logprobs-b4", op="logprobs", B=4, n=5, V=1000, K=5, dtype="f32", tempered=False),
        # The emitted tokens of one cycle of 128 requests over a 32000-token vocabulary.
        dict(name="logprobs-b128", op="logprobs", B=128, n=8, V=32000, K=20, dtype="bf16",
             tempered=True),
        # 256 requests over a large vocabulary.
        dict(name="logprobs-b256", op="logprobs", B=256, n=8, V=128256, K=8, dtype="bf16",
             tempered=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attention", "attention", "logprobs"])
    if op == "tables":
        B = _log_int(rng, 1, 2048)
        return dict(op=op, B=B, page=rng.choice([16, 32, 64, 128]), max_len=_log_int(rng, 16, 8192),
                    max_new=_log_int(rng, 1, max(2, min(1024, 1024 * 2048 // B))),
                    finished=rng.choice([0.0, 0.1, 0.3]))
    if op == "append":
        T = _log_int(rng, 1, 65553)
        D = rng.choice([64, 128, 256])
        H = rng.choice([h for h in (1, 2, 3, 4, 8) if h * D <= 1024])
        return dict(op=op, T=T, H=H, D=D, page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]) if T <= 30000 else "bf16",
                    fused=rng.random() < 0.5, skipped=rng.choice([0.0, 0.1]))
    if op == "attention":
        kind = rng.choice(["one", "block", "tree"])
        B = _log_int(rng, 1, 128)
        D = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([h for h in (1, 2, 4, 8) if h * D <= 1024])
        group = rng.choice([1, 2, 3, 4, 6, 8])
        max_new = 1 if kind == "one" else rng.randint(2, 17) if kind == "block" else rng.randint(4, 33)
        room = 128 * 8192 // B                       # tokens of a request, padded
        max_len = _log_int(rng, max_new + 1, max(max_new + 2, min(131072, room)))
        if kind != "one":                            # rows cost products: keep below the largest
            max_len = max(max_new + 1, min(max_len, room * 32 // (max_new * group)))
        return dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), kind=kind, max_new=max_new,
                    min_len=max_new, max_len=max_len)
    V = _log_int(rng, 16, 151936)
    rows = _log_int(rng, 1, max(2, min(2048, 256 * 8 * 64000 // V)))
    n = min(rows, rng.randint(1, 16))
    return dict(op=op, B=max(1, rows // n), n=n, V=V, K=min(V, rng.choice([0, 1, 5, 8, 20, 32])),
                dtype=rng.choice(["bf16", "bf16", "f32"]), tempered=rng.random() < 0.5)


# ------------------------------------------------------------------ the inputs

def _lengths(case, rng):
    """Lengths and new tokens of each request of an attention case, on the host."""
    B, new = case["B"], case["max_new"]
    if case["kind"] == "block":
        # verify lengths 1..max_new - 1 and the anchor: the same ones in another order
        n = rng.permutation(2 + np.arange(B) % max(1, new - 1))
    else:
        n = np.full(B, new)
    kv = np.maximum(n, rng.integers(case["min_len"], case["max_len"] + 1, B))
    return n.astype(np.int32), kv.astype(np.int32)


def _host_rng(case, seed):
    return np.random.default_rng([seed & 0x7FFFFFFF] + [ord(ch) for ch in case["op"]])


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


def _random_cache(gen, pages, H, page, D, k_scale, v_scale):
    """A cache of random keys (channels of different size) and values."""
    cache = torch.empty((pages, H, page // 16, 18 * D), dtype=torch.uint8, device=DEV)
    kc, ks, vc, vs = _parts(cache, D)
    channel = torch.exp(0.5 * torch.randn((H, D), generator=gen, device=DEV))
    step = max(1, (1 << 26) // (H * page * D))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        k = torch.randn((n, page // 16, 16, H, D), generator=gen, device=DEV) * channel
        v = torch.randn((n, page // 16, 16, H, D), generator=gen, device=DEV)
        kc[at:at + n], ks[at:at + n], _ = _to_4bit(k, k_scale)
        vc[at:at + n], vs[at:at + n], _ = _to_4bit(v, v_scale)
    return cache


def _prepare_tables(case, rng, gen):
    B, P = case["B"], case["page"]
    gamma = max(1, min(16, case["max_new"] - 1))
    seq = rng.integers(0, case["max_len"] + 1, B)
    accept = rng.integers(-1, gamma + 1, B)          # -1: nothing was kept of the last block
    new = rng.integers(0, case["max_new"] + 1, B)
    new[rng.random(B) < case["finished"]] = -1
    # pages held: those of the length and of the last, partly rejected, block
    held = -(-(seq + gamma + 1) // P)
    need = -(-(seq + accept + 1 + np.maximum(new, 0)) // P)
    stride = -(-(case["max_len"] + 17 + case["max_new"]) // P)
    pages = B * stride
    free = int(np.maximum(need - held, 0).sum())     # enough, or a pool that runs out
    free = min(pages - int(held.sum()), free + 7 if rng.random() < 0.75 else free * 3 // 4)
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((B, stride), -1, np.int32)
    table[np.arange(stride)[None, :] < held[:, None]] = perm[:held.sum()]
    head = int(rng.integers(0, 10 * pages))
    ring = np.full(pages, -1, np.int32)
    ring[(head + np.arange(free)) % pages] = perm[held.sum():held.sum() + free]
    rows = B * case["max_new"]

    def i32(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)

    def empty(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype, device=DEV)
    return dict(page=P, seq_len=i32(seq), accept_len=i32(accept), new_len=i32(new),
                num_blocks=i32(held), ring_pos=torch.tensor([head, head + free], device=DEV),
                free_ring=i32(ring), block_table=i32(table), seq_len_out=empty(B), kv_len=empty(B),
                num_blocks_out=empty(B), ring_pos_out=empty(2, dtype=torch.int64),
                row_ptr=empty(B + 1), slots=empty(rows), positions=empty(rows), status=empty(4))


def _prepare_append(case, rng, gen):
    T, H, D, P = case["T"], case["H"], case["D"], case["page"]
    dt = DTYPES[case["dtype"]]
    channel = torch.exp(0.5 * torch.randn((H, D), generator=gen, device=DEV))
    if case["fused"]:                                # [query heads | key heads | value heads]
        qkv = torch.empty((T, 6 * H, D), dtype=dt, device=DEV)
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device=DEV))
        k, v = qkv[:, 4 * H:5 * H], qkv[:, 5 * H:]
        k.mul_(channel.to(dt))
    else:
        k = (torch.randn((T, H, D), generator=gen, device=DEV) * channel).to(dt)
        v = torch.randn((T, H, D), generator=gen, device=DEV).to(dt)
    pages = -(-T // P) + 3
    slots = rng.permutation(pages * P)[:T] if T <= 4096 else None
    if slots is None:                                # prompts: whole pages in random order
        at = np.arange(T)
        slots = rng.permutation(pages)[at // P] * P + at % P
    slots[rng.random(T) < case["skipped"]] = -1
    cache = torch.zeros((pages, H, P // 16, 18 * D), dtype=torch.uint8, device=DEV)
    return dict(page=P, D=D, k=k, v=v, slots=torch.from_numpy(slots.astype(np.int32)).to(DEV),
                cache=cache, k_scale=K_SCALE, v_scale=V_SCALE,
                k_stored=torch.empty((T, H, D), dtype=dt, device=DEV),
                v_stored=torch.empty((T, H, D), dtype=dt, device=DEV),
                status=torch.zeros(4, dtype=torch.int32, device=DEV))


def _prepare_attention(case, rng, gen):
    B, P, D, Hkv, Hq = case["B"], case["page"], case["D"], case["Hkv"], case["Hq"]
    n, kv = _lengths(case, rng)
    blocks = -(-kv // P)
    pages = int(blocks.sum()) + 5
    table = np.full((B, -(-case["max_len"] // P)), -1, np.int32)
    table[np.arange(table.shape[1])[None, :] < blocks[:, None]] = rng.permutation(pages)[:blocks.sum()]
    ptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T = int(ptr[-1])
    mask = None
    if case["kind"] == "tree":                       # row i of a request sees itself and its ancestors
        words = -(-case["max_new"] // 32)
        bits = np.zeros((B, case["max_new"], words), np.uint32)
        for i in range(case["max_new"]):
            if i:
                bits[:, i] = bits[np.arange(B), rng.integers(max(0, i - 6), i, B)]
            bits[:, i, i // 32] |= np.uint32(1 << (i % 32))
        mask = torch.from_numpy(bits.reshape(T, words).view(np.int32)).to(DEV)
    k_scale, v_scale = K_SCALE, V_SCALE
    dt = DTYPES[case["dtype"]]
    return dict(page=P, D=D, Hq=Hq, Hkv=Hkv, B=B, max_new=int(n.max()), max_kv=int(kv.max()), mask=mask,
                softmax_scale=1.0 / math.sqrt(D), k_scale=k_scale, v_scale=v_scale,
                q=torch.randn((T, Hq, D), generator=gen, device=DEV).to(dt),
                cache=_random_cache(gen, pages, Hkv, P, D, k_scale, v_scale),
                block_table=torch.from_numpy(table).to(DEV), kv_len=torch.from_numpy(kv).to(DEV),
                row_ptr=torch.from_numpy(ptr).to(DEV), out=torch.empty((T, Hq, D), dtype=dt, device=DEV),
                lse=torch.empty((T, Hq), dtype=torch.float32, device=DEV),
                status=torch.zeros(4, dtype=torch.int32, device=DEV))


def _prepare_logprobs(case, rng, gen):
    B, n, V, K = case["B"], case["n"], case["V"], case["K"]
    logits = torch.empty((B, n, V), dtype=DTYPES[case["dtype"]], device=DEV)
    for b in range(0, B, 64):
        logits[b:b + 64] = 3.0 * torch.randn(logits[b:b + 64].shape, generator=gen, device=DEV)
    # the tokens of a verified block: the accepted ones and the last, then -1
    emitted = rng.integers(1, n + 1, B)
    tokens = rng.integers(0, V, (B, n))
    best = rng.random((B, n)) < 0.5                  # likely tokens, as a sampler's are
    tokens = np.where(best, logits.argmax(-1).cpu().numpy(), tokens)
    tokens[np.arange(n)[None, :] >= emitted[:, None]] = -1
    t = rng.choice([0.6, 0.7, 1.0], B).astype(np.float32)
    return dict(K=K, logits=logits, tokens=torch.from_numpy(tokens.astype(np.int32)).to(DEV),
                temperature=torch.from_numpy(t).to(DEV) if case["tempered"] else None,
                logprob=torch.empty((B, n), dtype=torch.float32, device=DEV),
                entropy=torch.empty((B, n), dtype=torch.float32, device=DEV),
                top_ids=torch.empty((B, n, K), dtype=torch.int32, device=DEV) if K else None,
                top_logprobs=torch.empty((B, n, K), dtype=torch.float32, device=DEV) if K else None,
                status=torch.zeros(4, dtype=torch.int32, device=DEV))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    make = dict(tables=_prepare_tables, append=_prepare_append, attention=_prepare_attention,
                logprobs=_prepare_logprobs)[case["op"]]
    return dict(make(case, _host_rng(case, seed), gen), op=case["op"])


# ------------------------------------------------------------- the plain forms

def _plain_tables(s):
    P, stride, pages = s["page"], s["block_table"].shape[1], s["free_ring"].numel()
    B, max_rows = s["seq_len"].numel(), s["slots"].numel()
    dev = s["seq_len"].device
    index = torch.arange(B, device=dev)
    base = torch.where(s["new_len"] < 0, torch.zeros_like(s["seq_len"]), s["seq_len"] + s["accept_len"] + 1)
    new = s["new_len"].clamp(min=0)
    held, free = s["num_blocks"], s["ring_pos"][1] - s["ring_pos"][0]
    # requests are served in order; from the first that finds no room on, none appends
    ask = ((base + new + P - 1) // P - held).clamp(min=0)
    full = (ask.cumsum(0) > free) | (new.cumsum(0) > max_rows)
    first = torch.where(full & (new > 0), index, B).amin()
    new = torch.where(index >= first, 0, new)
    kv = base + new
    need = (kv + P - 1) // P
    ask, back = (need - held).clamp(min=0), (held - need).clamp(min=0)
    ask_end, back_end = ask.cumsum(0), back.cumsum(0)
    column = torch.arange(stride, device=dev)
    head, tail = s["ring_pos"][0], s["ring_pos"][1]
    take = (head + (ask_end - ask).unsqueeze(1) + (column - held.unsqueeze(1))) % pages
    fresh = (column >= held.unsqueeze(1)) & (column < need.unsqueeze(1))
    table = torch.where(fresh, s["free_ring"][take.clamp(min=0)], s["block_table"])
    gone = (column >= need.unsqueeze(1)) & (column < held.unsqueeze(1))
    give = (tail + (back_end - back).unsqueeze(1) + (column - need.unsqueeze(1))) % pages
    ring = s["free_ring"].clone()
    ring[give[gone]] = s["block_table"][gone]
    ptr = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), new.cumsum(0)])
    row = torch.arange(max_rows, device=dev)
    who = torch.searchsorted(ptr[1:].contiguous(), row, right=True).clamp(max=B - 1)
    live = row < ptr[-1]
    position = torch.where(live, base[who] + row - ptr[who], 0)
    slot = table[who, position // P] * P + position % P
    none = torch.full((), -1, dtype=torch.int32, device=dev)
    return dict(seq_len=base.int(), kv_len=kv.int(), num_blocks=need.int(),
                ring_pos=torch.stack([head + ask_end[-1], tail + back_end[-1]]), free_ring=ring,
                block_table=table, row_ptr=ptr.int(), slots=torch.where(live, slot.int(), none),
                positions=torch.where(live, position.int(), none))


def _plain_append(s):
    P, D = s["page"], s["D"]
    kc, ks, vc, vs = _parts(s["cache"], D)
    live = s["slots"] >= 0
    slot = s["slots"][live].long()
    at = (slot // P, slot % P // 16, slot % 16)
    k, v = s["k"].float(), s["v"].float()
    codes, scales, k_val = _to_4bit(k, s["k_scale"])
    kc[at], ks[at] = codes[live], scales[live]
    codes, scales, v_val = _to_4bit(v, s["v_scale"])
    vc[at], vs[at] = codes[live], scales[live]
    keep = live[:, None, None]
    zero = torch.zeros((), device=DEV)
    return dict(k_stored=torch.where(keep, k_val, zero).to(s["k"].dtype),
                v_stored=torch.where(keep, v_val, zero).to(s["v"].dtype))


def _plain_attention(s):
    P, D, B, Hkv, n, L = s["page"], s["D"], s["B"], s["Hkv"], s["max_new"], s["max_kv"]
    G = s["Hq"] // Hkv
    pos = torch.arange(L, device=DEV)
    page = s["block_table"][:, pos // P].clamp(min=0)
    at = (page, (pos % P // 16).expand(B, L), (pos % 16).expand(B, L))
    kc, ks, vc, vs = _parts(s["cache"], D)
    there = pos < s["kv_len"][:, None]
    k = _from_4bit(kc[at], ks[at], s["k_scale"])                   # [B, L, Hkv, D]
    row = torch.arange(n, device=DEV)
    ptr = s["row_ptr"]
    fresh = ptr[1:] - ptr[:-1]
    rows = (ptr[:-1, None] + row).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["softmax_scale"]
    del k
    ctx = (s["kv_len"] - fresh)[:, None, None]
    if s["mask"] is None:
        seen = pos <= ctx + row[:, None]
    else:
        tail = (pos - ctx).expand(B, n, L)
        word = s["mask"][rows].gather(-1, (tail.clamp(0, 32 * s["mask"].shape[1] - 1) // 32))
        seen = (tail < 0) | ((word >> (tail.clamp(min=0) % 32)) & 1).bool()
    seen = (seen & there[:, None]).repeat(1, G, 1)[:, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    total = e.sum(-1, keepdim=True)
    v = _from_4bit(vc[at], vs[at], s["v_scale"])
    v = torch.where(there[..., None, None], v, 0.0).permute(0, 2, 1, 3)
    y = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total)).view(B, Hkv, G, n)
    y = y.view(B, Hkv, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, s["Hq"], D)
    live = row < fresh[:, None]
    return dict(out=y[live].to(s["q"].dtype), lse=lse.permute(0, 3, 1, 2).reshape(B, n, s["Hq"])[live])


def _plain_logprobs(s):
    K, V = s["K"], s["logits"].shape[-1]
    x = s["logits"].float()
    if s["temperature"] is not None:
        x = x / s["temperature"][:, None, None]
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    total = e.sum(-1)
    log_total = torch.log(total)
    entropy = log_total - (e * d).sum(-1) / total
    del e
    live = s["tokens"] >= 0
    none = torch.full((), math.nan, device=DEV)
    given = d.gather(-1, s["tokens"].clamp(min=0).long().unsqueeze(-1)).squeeze(-1) - log_total
    out = dict(logprob=torch.where(live, given, none), entropy=torch.where(live, entropy, none))
    if K:
        # one key of value, then lowest index: whole numbers in the order of the 32-bit logits
        raw = s["logits"].float().view(torch.int32)
        raw = torch.where(raw == -2 ** 31, 0, raw)
        order = torch.where(raw < 0, raw ^ 0x7FFFFFFF, raw).long()
        key = order * 2 ** 24 + (2 ** 24 - 1 - torch.arange(V, device=DEV))
        ids = (2 ** 24 - 1 - torch.topk(key, K, dim=-1).values % 2 ** 24).int()
        top = d.gather(-1, ids.long()) - log_total.unsqueeze(-1)
        out["top_ids"] = torch.where(live[..., None], ids, -1)
        out["top_logprobs"] = torch.where(live[..., None], top, none)
    return out


# -------------------------------------------------------------- the operators

def _own_tables(s):
    from speculative_decoding_draft_04_gb300 import _lib
    _lib.spec_block_tables(s["seq_len"], s["accept_len"], s["new_len"], s["num_blocks"], s["ring_pos"],
                           s["free_ring"], s["block_table"], s["seq_len_out"], s["kv_len"],
                           s["num_blocks_out"], s["ring_pos_out"], s["row_ptr"], s["slots"],
                           s["positions"], s["status"], s["page"])
    return dict(seq_len=s["seq_len_out"], kv_len=s["kv_len"], num_blocks=s["num_blocks_out"],
                ring_pos=s["ring_pos_out"], free_ring=s["free_ring"], block_table=s["block_table"],
                row_ptr=s["row_ptr"], slots=s["slots"], positions=s["positions"])


def _own_append(s):
    from speculative_decoding_draft_04_gb300 import _lib
    _lib.spec_cache_append(s["k"], s["v"], s["slots"], s["cache"], s["status"], s["k_scale"], s["v_scale"],
                           k_stored=s["k_stored"], v_stored=s["v_stored"])
    return dict(k_stored=s["k_stored"], v_stored=s["v_stored"])


def _own_attention(s):
    from speculative_decoding_draft_04_gb300 import _lib
    if "workspace" not in s:
        s["workspace"] = torch.empty(_lib.spec_cache_attention_workspace_bytes(s["Hq"], s["Hkv"], s["D"]),
                                     dtype=torch.uint8, device=DEV)
    _lib.spec_cache_attention(s["q"], s["cache"], s["block_table"], s["kv_len"], s["row_ptr"], s["out"],
                              s["status"], s["workspace"], s["softmax_scale"], s["k_scale"], s["v_scale"],
                              tree_mask=s["mask"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _own_logprobs(s):
    from speculative_decoding_draft_04_gb300 import _lib
    if "workspace" not in s:
        B, n, V = s["logits"].shape
        s["workspace"] = torch.empty(_lib.spec_logprobs_workspace_bytes(B * n, V, s["K"]),
                                     dtype=torch.uint8, device=DEV)
    _lib.spec_logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], s["status"], s["workspace"],
                       temperature=s["temperature"], top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
    out = dict(logprob=s["logprob"], entropy=s["entropy"])
    if s["K"]:
        out.update(top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
    return out


def run(state):
    if own:
        return dict(tables=_own_tables, append=_own_append, attention=_own_attention,
                    logprobs=_own_logprobs)[state["op"]](state)
    return dict(tables=_plain_tables, append=_plain_append, attention=_plain_attention,
                logprobs=_plain_logprobs)[state["op"]](state)


# ------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "tables":
        # four words a request in and four out, a slot and a position a row (half of them are live
        # on average), a page id read and written for each page that changes hands
        rows = case["B"] * case["max_new"] / 2 * (1 - case["finished"])
        pages = rows / case["page"]
        return dict(bytes=32 * case["B"] + 8 * case["B"] * case["max_new"] + 8 * pages, flops=0)
    if op == "append":
        n = case["T"] * case["H"] * case["D"] * 2
        return dict(bytes=n * (2 * SIZES[case["dtype"]]) + n * 9 / 16 + 4 * case["T"], flops=4 * n)
    if op == "attention":
        # the mean over the lengths' distribution: every key and value once, the rows in and out
        new = case["max_new"] if case["kind"] != "block" else (min(2, case["max_new"]) + case["max_new"]) / 2
        tokens = case["B"] * (case["min_len"] + case["max_len"]) / 2
        rows = case["B"] * new * case["Hq"]
        return dict(bytes=tokens * case["Hkv"] * case["D"] * 9 / 8 + rows * case["D"] * 2 * SIZES[case["dtype"]],
                    flops=4 * tokens * new * case["Hq"] * case["D"])
    rows = case["B"] * (case["n"] + 1) / 2           # the emitted tokens' rows
    return dict(bytes=rows * case["V"] * SIZES[case["dtype"]] + case["B"] * case["n"] * (12 + 8 * case["K"]),
                flops=6 * rows * case["V"])


# ----------------------------------------------------------------- in 64 bits

def _exact_levels(y):
    """The nearest 4-bit level of |y| in 64 bits, ties to the even code."""
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=y.device)
    hi = torch.searchsorted(levels, y.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    up, down = levels[hi] - y, y - levels[lo]
    return levels[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]


def _exact_append(s):
    def store(x, g):
        out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        for at in range(0, x.shape[0], 4096):
            z = x[at:at + 4096].double().unflatten(-1, (-1, 16))
            t = (z.abs().amax(-1) / (6.0 * g)).clamp(max=448.0)
            step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
            r = (torch.round(t / step) * step * g).unsqueeze(-1)
            y = _exact_levels((z.abs() / torch.where(r > 0, r, 1.0)).clamp(max=6.0)) * r
            out[at:at + 4096] = (torch.sign(z) * y).flatten(-2)
        out[s["slots"] < 0] = 0.0
        return out
    return dict(k_stored=store(s["k"], s["k_scale"]), v_stored=store(s["v"], s["v_scale"]))


def _exact_attention(s):
    D, P, Hkv = s["D"], s["page"], s["Hkv"]
    G = s["Hq"] // Hkv
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)

    def value(codes, scales, g):
        c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
        x = torch.where(c >= 8, -1.0, 1.0).double() * levels[c % 8]
        e, f = scales.long() // 8 % 16, (scales.long() % 8).double()
        sc = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2(e.double() - 7))
        return x * sc.repeat_interleave(16, -1) * g
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    ptr, kv = s["row_ptr"].tolist(), s["kv_len"].tolist()
    for b in range(s["B"]):
        n, L = ptr[b + 1] - ptr[b], kv[b]
        pages = s["block_table"][b, :-(-L // P)].long()
        see = torch.ones((n, L), dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            see = torch.tril(see, diagonal=L - n)
        else:
            words = s["mask"][ptr[b]:ptr[b + 1]].long() & 0xFFFFFFFF
            bits = (words[:, :, None] >> torch.arange(32, device=DEV)) & 1
            see[:, L - n:] = bits.flatten(1)[:, :n].bool()
        for h in range(Hkv):
            block = s["cache"][pages, h].flatten(0, 1)             # [blocks of 16 tokens, 18 D]
            k = value(block[:, :8 * D].reshape(-1, D // 2), block[:, 8 * D:9 * D].reshape(-1, D // 16),
                      s["k_scale"])[:L]
            v = value(block[:, 9 * D:17 * D].reshape(-1, D // 2), block[:, 17 * D:].reshape(-1, D // 16),
                      s["v_scale"])[:L]
            q = s["q"][ptr[b]:ptr[b + 1], h * G:(h + 1) * G].double()
            x = (q.reshape(n * G, D) @ k.T).view(n, G, L) * s["softmax_scale"]
            x = x.masked_fill(~see[:, None], -math.inf)
            lse[ptr[b]:ptr[b + 1], h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            out[ptr[b]:ptr[b + 1], h * G:(h + 1) * G] = (torch.softmax(x, -1).view(n * G, L) @ v).view(n, G, D)
    return dict(out=out, lse=lse)


def _exact_logprobs(s):
    B, n, V = s["logits"].shape
    shape = dict(dtype=torch.float64, device=DEV)
    logprob, entropy = torch.full((B, n), math.nan, **shape), torch.full((B, n), math.nan, **shape)
    out = dict(logprob=logprob, entropy=entropy)
    if s["K"]:
        out["top_ids"] = None
        out["top_logprobs"] = torch.full((B, n, s["K"]), math.nan, **shape)
    for b in range(B):
        live = s["tokens"][b] >= 0
        x = s["logits"][b][live].double()
        if s["temperature"] is not None:
            x = x / s["temperature"][b].double()
        logp = torch.log_softmax(x, -1)
        logprob[b, live] = logp.gather(-1, s["tokens"][b][live].long()[:, None])[:, 0]
        entropy[b, live] = -(torch.exp(logp) * logp).sum(-1)
        if s["K"]:
            out["top_logprobs"][b, live] = torch.sort(logp, dim=-1, descending=True).values[:, :s["K"]]
    return out


def exact(case, seed):
    if case["op"] == "tables":                       # whole numbers
        return None
    return dict(append=_exact_append, attention=_exact_attention,
                logprobs=_exact_logprobs)[case["op"]](prepare(case, seed))
