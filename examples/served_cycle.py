"""A few cycles of a server with a small random target model on one GPU:
prompts into the paged 4-bit cache, then draft, target pass over the block,
verification and log probabilities of the emitted tokens.

    python examples/served_cycle.py [--requests 8] [--cycles 4]

The model is untrained: what it emits means nothing, but every step is the one
that a server makes.  Its projections are plain matrix products; everything
else of a cycle is a call of the library.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch

from speculative_decoding_draft_04_gb300 import engine, workloads


class Target:
    """Layers of attention over the cache with residual sums, random weights."""

    def __init__(self, V, width, layers, Hq, Hkv, D, gen):
        def w(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") * shape[0] ** -0.5).bfloat16()
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.embed = (torch.randn((V, width), generator=gen, device="cuda")).bfloat16()
        self.qkv = [w(width, (Hq + 2 * Hkv) * D) for _ in range(layers)]
        self.proj = [w(Hq * D, width) for _ in range(layers)]
        self.head = w(width, V)

    def __call__(self, tokens, c, last=None):
        """Logits of the packed rows (of the rows ``last`` only, where given)."""
        x = self.embed[tokens.long()]
        T, Hq, Hkv, D = x.shape[0], self.Hq, self.Hkv, self.D
        for i, (wi, wo) in enumerate(zip(self.qkv, self.proj)):
            y = (torch.nn.functional.rms_norm(x, x.shape[1:]) @ wi).view(T, Hq + 2 * Hkv, D)
            o = torch.zeros((T, Hq, D), dtype=x.dtype, device=x.device)
            engine.attend(c, i, y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], o)
            x = x + o.view(T, Hq * D) @ wo
        x = x if last is None else x[last]
        return torch.nn.functional.rms_norm(x, x.shape[1:]) @ self.head


def serve(requests=8, cycles=4, prompt=100, gamma=7, V=32000, width=512, layers=2, Hq=16, Hkv=4, D=64,
          page_size=32, top=5, seed=0, pages=None):
    """Per cycle: tokens emitted (int32 [B, gamma + 1], -1 padded), their log
    probabilities, and the cache with the lengths of its requests.  pages: of
    the pool, by default enough for every request; a request that finds none
    for its block emits nothing in that cycle and goes on when there are."""
    gen = torch.Generator("cuda").manual_seed(seed)
    B, n = requests, gamma + 1
    model = Target(V, width, layers, Hq, Hkv, D, gen)
    w = workloads.make_workload(workloads.config("C1", B=B, V=V, gamma=gamma, target=("normal", 0.5),
                                               noise=("fixed", 0.5)))
    d = engine.DeviceWorkload.from_workload(w)
    b = engine.Buffers.for_workload(d)
    l = engine.DeviceLogprobs.allocate(B, n, V, K=top)
    most = prompt + B + (cycles + 1) * n                      # tokens of the longest request
    rows = B * prompt + B * (B - 1) // 2
    c = engine.DeviceCache.allocate(B, layers, Hq, Hkv, D, page_size, pages or B * -(-most // page_size), most,
                                    max(rows, B * n), [0.01] * layers, [0.01] * layers)
    # prompts, one token longer from request to request; the last token of each
    # becomes the first anchor
    held = torch.arange(prompt, prompt + B, dtype=torch.int32, device="cuda")
    tokens = torch.randint(0, V, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    engine.make_room(c, held)
    first = model(tokens, c, last=(c.row_ptr[1:] - 1).long())
    d.anchor.copy_(first.argmax(-1))
    block = torch.full((B,), n, dtype=torch.int32, device="cuda")

    row = torch.arange(B * n, device="cuda")

    def target_pass(d, b, c, stream):
        # packed row r is token r - row_ptr[i] of the i-th request's block; a
        # request without pages for its block has no rows (those beyond
        # row_ptr[B] belong to nobody)
        ptr = c.row_ptr.long()
        who = torch.searchsorted(ptr[1:], row, right=True).clamp(max=B - 1)
        fed = torch.cat([d.anchor[:, None], b.draft_tokens], 1)
        logits = model(fed[who, (row - ptr[who]).clamp(max=n - 1)], c)
        at = (ptr[:-1, None] + row[:n]).clamp(max=B * n - 1)
        d.target.copy_(logits[at])

    kept, out = held - 1, []
    for _ in range(cycles):
        for u in (d.u_draft, d.u_accept, d.u_final):
            u.uniform_(generator=gen)
        engine.served_cycle(d, b, c, l, target_pass, block, kept)
        kept = b.accept_len.clone()
        newest = b.out_tokens.gather(1, kept.clamp(min=0)[:, None].long())[:, 0]
        d.anchor.copy_(torch.where(kept < 0, d.anchor, newest))
        out.append((b.out_tokens.clone(), l.logprob.clone()))
    words = [engine.status_words(t)[0] for t in (b.dstatus, b.vstatus, c.status, l.status)]
    words[2] &= ~256                                          # pages that were not there
    if any(words):
        raise RuntimeError(f"status words {words}")
    return out, c


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--cycles", type=int, default=4)
    a = p.parse_args()
    out, c = serve(a.requests, a.cycles)
    for i, (tokens, lp) in enumerate(out):
        live = tokens >= 0
        print(f"cycle {i}: {int(live.sum())} tokens emitted, mean log probability "
              f"{float(lp[live].mean()):.3f}; request 0: {tokens[0][live[0]].tolist()}")
    print("tokens held:", c.seq_len[c.newest].tolist(), "pages:", c.num_blocks[c.newest].tolist())


if __name__ == "__main__":
    main()
