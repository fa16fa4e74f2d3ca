"""Shared helpers of the serving operators' GPU tests: random inputs on the host and the calls."""
import numpy as np

from oracle import serving as S


def lib():
    from speculative_decoding_draft_04_gb300 import _lib
    return _lib


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return t.to("cuda") if dtype is None else t.to("cuda").to(dtype)


def status(st) -> int:
    return int(st[0].item()) & 0xFFFFFFFF


def new_status():
    import torch
    return torch.zeros(4, dtype=torch.int32, device="cuda")


def storage(torch, dtype):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def rounded(a, dtype):
    """float64 values of a as the storage type holds them."""
    import torch
    return torch.from_numpy(np.asarray(a, np.float32)).to(storage(torch, dtype)).double().numpy()


# ------------------------------------------------------------- attention

class Paged:
    """A random paged 4-bit cache on the host with its requests."""

    def __init__(self, rng, lens, news, Hq, Hkv, D, page, dtype, tree=None, k_scale=0.011, v_scale=0.003,
                 junk=True, q_size=1.0, extra_pages=3):
        B = len(lens)
        self.lens, self.news = np.asarray(lens, np.int32), np.asarray(news, np.int32)
        self.Hq, self.Hkv, self.D, self.page, self.dtype = Hq, Hkv, D, page, dtype
        self.k_scale, self.v_scale = float(np.float32(k_scale)), float(np.float32(v_scale))
        blocks = -(-self.lens // page)
        pages = int(blocks.sum()) + extra_pages
        order = rng.permutation(pages)
        self.table = np.full((B, max(1, int(blocks.max())) + 1), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :blocks[b]] = order[at:at + blocks[b]]
            at += blocks[b]
        # bytes of tokens that nobody wrote are arbitrary, scale bytes that mean no number included
        self.cache = rng.integers(0, 256, (pages, Hkv, page // 16, 18 * D), dtype=np.uint8) if junk \
            else np.zeros((pages, Hkv, page // 16, 18 * D), np.uint8)
        for which in (0, 1):
            (c0, c1), (s0, s1) = S.block_parts(D)[2 * which:2 * which + 2]
            for b in range(B):
                for t0 in range(0, int(self.lens[b]), 16):
                    n = min(16, int(self.lens[b]) - t0)
                    blk = self.cache[self.table[b, t0 // page], :, t0 % page // 16]
                    code = rng.integers(0, 256, (Hkv, n, D // 2), dtype=np.uint8)
                    sc = rng.integers(0x40, 0x68, (Hkv, n, D // 16), dtype=np.uint8)
                    blk[:, c0:c0 + n * (D // 2)] = code.reshape(Hkv, -1)
                    blk[:, s0:s0 + n * (D // 16)] = sc.reshape(Hkv, -1)
        self.ptr = np.concatenate([[0], np.cumsum(self.news)]).astype(np.int32)
        self.T = int(self.ptr[-1])
        self.q = rounded(rng.normal(size=(self.T, Hq, D)) * q_size, dtype)
        self.mask = None
        if tree is not None:
            self.mask = tree(rng, self)

    def run(self, torch, scale, stream=None, out=None, q=None, row_ptr=None, T=None, lse=True):
        L = lib()
        st = new_status()
        dt = storage(torch, self.dtype)
        q = dev(self.q, dt) if q is None else q
        T = q.shape[0]
        out = torch.full((T, self.Hq, self.D), 7.0, dtype=dt, device="cuda") if out is None else out
        lse = torch.full((T, self.Hq), 7.0, dtype=torch.float32, device="cuda") if lse else None
        ws = torch.full((L.spec_cache_attention_workspace_bytes(self.Hq, self.Hkv, self.D),), 0xA5,
                        dtype=torch.uint8, device="cuda")
        L.spec_cache_attention(q, dev(self.cache), dev(self.table), dev(self.lens),
                               dev(self.ptr) if row_ptr is None else row_ptr, out, st, ws, scale,
                               self.k_scale, self.v_scale,
                               tree_mask=None if self.mask is None else dev(self.mask.view(np.int32)),
                               lse=lse, stream=stream)
        torch.cuda.synchronize()
        return (out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy(), status(st))

    def oracle(self, scale, requests=None):
        """out, lse, the tolerance of out and of lse (see test_cache_attention_gpu)."""
        G = self.Hq // self.Hkv
        out = np.zeros((self.T, self.Hq, self.D))
        lse = np.zeros((self.T, self.Hq))
        tol_o, tol_l = np.zeros_like(out), np.zeros_like(lse)
        half = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -22
        prob = 2.0 ** -11 if self.dtype == "bf16" else 2.0 ** -20
        for b in range(len(self.lens)) if requests is None else requests:
            n, L = int(self.news[b]), int(self.lens[b])
            r = slice(self.ptr[b], self.ptr[b + 1])
            see = S.visible(n, L, None if self.mask is None else self.mask[r])
            for h in range(self.Hkv):
                k = S.read_tokens(self.cache, self.table[b], h, L, self.D, 0, self.k_scale)
                v = S.read_tokens(self.cache, self.table[b], h, L, self.D, 1, self.v_scale)
                for i in range(h * G, (h + 1) * G):
                    o, l, absv, big = S.attention(self.q[r, i], k, v, see, scale)
                    out[r, i], lse[r, i] = o, l
                    x = 2.0 ** -18 * big[:, None]          # error of a score
                    tol_o[r, i] = half * np.abs(o) + (prob + 2 * x + 2.0 ** -15) * absv + 1e-30
                    tol_l[r, i] = x[:, 0] + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(l), l, 0)))
        return out, lse, tol_o, tol_l


def tree_of(max_back=4, empty=False):
    """Ancestor masks of random trees over each request's new rows."""
    def make(rng, p):
        words = -(-int(p.news.max()) // 32)
        mask = np.zeros((p.T, words), np.uint32)
        for b in range(len(p.news)):
            for i in range(p.news[b]):
                row = p.ptr[b] + i
                if i:
                    mask[row] = mask[p.ptr[b] + rng.integers(max(0, i - max_back), i)]
                mask[row, i // 32] |= np.uint32(1 << (i % 32))
            if empty:
                mask[p.ptr[b] + p.news[b] // 2] = 0
        return mask
    return make
