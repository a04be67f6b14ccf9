"""Inputs and 64-bit references of attention through a sliding window with sinks and of trees of drafted tokens (test
infrastructure: numpy and torch, no library code)."""
import numpy as np
import torch

SB = 16


def window_sees(L, n, window, sinks):
    """bool [n, L]: the keys that the last n queries of L tokens see."""
    p = np.arange(L - n, L)[:, None]
    j = np.arange(L)[None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def tree_sees(L, n, mask):
    """bool [n, L] from the nodes' mask rows, int32 [n, words]."""
    sees = np.zeros((n, L), bool)
    sees[:, :L - n] = True
    bits = np.unpackbits(np.ascontiguousarray(mask).view(np.uint8), axis=1, bitorder="little")[:, :n]
    sees[:, L - n:] = bits.astype(bool) & (np.arange(n)[None] <= np.arange(n)[:, None])
    return sees


def random_trees(new, words, rng, noise=True):
    """int32 [rows, words]: each node sees itself and its ancestors; noise: bits of later nodes and past the tree too,
    which do not count."""
    rows = []
    for n in new:
        m = np.zeros((n, 32 * words), np.uint8)
        for i in range(n):
            if i:
                m[i] = m[rng.integers(max(0, i - 6), i)]
            m[i, i] = 1
        if noise:
            late = np.arange(32 * words)[None] > np.arange(n)[:, None]
            m |= (late & (rng.random(m.shape) < 0.3)).astype(np.uint8)
        rows.append(np.packbits(m, axis=1, bitorder="little"))
    return np.ascontiguousarray(np.concatenate(rows)).view(np.int32).reshape(-1, words)


class Problem:
    """A paged cache of a batch whose row b of `sees` (a bool [n, L] each) says what its queries see.  Pages that no
    query sees are not held (their table entries name no block); every other row and scale that no query sees holds
    what would spoil the result if it counted."""

    def __init__(self, cache, sees, Hq, Hkv, D, bs, seed, spread=1.0, bad=-1):
        rng = np.random.default_rng(seed)
        self.cache, self.sees, self.D, self.bs, self.Hq, self.Hkv = cache, sees, D, bs, Hq, Hkv
        self.lens, self.new = [s.shape[1] for s in sees], [s.shape[0] for s in sees]
        seen = [s.any(0) for s in sees]
        nblk = [-(-L // bs) for L in self.lens]
        held = [[p for p in range(m) if v[p * bs:(p + 1) * bs].any()] for m, v in zip(nblk, seen)]
        NB = sum(map(len, held)) + 3
        perm = rng.permutation(NB)
        self.bt = np.full((len(sees), max(max(nblk), 1)), bad, np.int32)
        live = np.zeros((NB, bs), bool)
        cur = 0
        for b, pages in enumerate(held):
            self.bt[b, pages] = perm[cur:cur + len(pages)]
            for i, p in enumerate(pages):
                v = seen[b][p * bs:(p + 1) * bs]
                live[perm[cur + i], :len(v)] = v
            cur += len(pages)
        g = torch.Generator().manual_seed(seed)
        shape = (NB, bs, Hkv, D)
        alive = torch.from_numpy(live)[:, :, None, None]
        self.scales = None
        if cache == "bf16":
            self.kc, self.vc = (torch.where(alive, torch.randn(shape, generator=g), float("nan")).bfloat16()
                                for _ in range(2))
            self.kd, self.vd = self.kc.double(), self.vc.double()
        elif cache == "fp8":
            codes = [torch.randint(0, 256, shape, generator=g).to(torch.uint8) for _ in range(2)]
            codes = [torch.where(c & 0x7F > 0x60, c & 0x9F, c) for c in codes]  # magnitudes up to 32
            self.kc, self.vc = (torch.where(alive, c, 0x7F) for c in codes)  # 0x7F: NaN
            self.scales = (torch.rand(Hkv, generator=g) * 0.1 + 0.02, torch.rand(Hkv, generator=g) * 0.1 + 0.02)
            self.kd, self.vd = (c.view(torch.float8_e4m3fn).double() * s.double()[:, None]
                                for c, s in zip((self.kc, self.vc), self.scales))
        else:
            self.kc, self.vc = (torch.where(alive, torch.randint(-127, 128, shape, generator=g), -128).to(torch.int8)
                                for _ in range(2))
            some = torch.from_numpy(live.reshape(NB, bs // SB, SB).any(2))[:, :, None, None]
            s = torch.exp((2 * torch.rand(NB, bs // SB, Hkv, 2, generator=g) - 1) * spread) * torch.tensor([0.01, 0.015])
            self.sc = torch.where(some, s, float("nan"))
            wide = self.sc.double().repeat_interleave(SB, 1)
            self.kd, self.vd = self.kc.double() * wide[..., 0:1], self.vc.double() * wide[..., 1:2]
        T = sum(self.new)
        self.q = torch.randn(T, Hq, D, generator=g).bfloat16()
        self.scale = D ** -0.5

    def cuda(self):
        """(q, caches, tables, lengths, offsets) on the GPU."""
        cache = [self.kc.cuda(), self.vc.cuda()]
        if self.cache == "fp8":
            cache += [s.cuda() for s in self.scales]
        elif self.cache == "int8":
            cache.append(self.sc.cuda())
        cu = np.concatenate([[0], np.cumsum(self.new)])
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
        return self.q.cuda(), cache, i32(self.bt), i32(self.lens), i32(cu)

    def want(self):
        """(out, mag): float64 [T, Hq, D], and the weighted mean of |v|; rows that see nothing are zeros."""
        T, G = self.q.shape[0], self.Hq // self.Hkv
        out, mag = (torch.zeros(T, self.Hq, self.D, dtype=torch.float64) for _ in range(2))
        r = 0
        for b, s in enumerate(self.sees):
            n, L = s.shape
            cols = np.nonzero(s.any(0))[0]
            if n and len(cols):
                at = torch.from_numpy(cols)
                page, row = torch.from_numpy(self.bt[b].astype(np.int64))[at // self.bs], at % self.bs
                k, v = self.kd[page, row], self.vd[page, row]                       # [cols, Hkv, D]
                hide = torch.from_numpy(~s[:, cols])
                q = self.q[r:r + n].double().view(n, self.Hkv, G, self.D)
                x = torch.einsum("nhgd,lhd->hgnl", q, k) * self.scale
                x = x.masked_fill(hide, float("-inf"))
                w = torch.where(hide.all(1)[:, None], 0.0, torch.softmax(x, -1))
                out[r:r + n] = torch.einsum("hgnl,lhd->nhgd", w, v).reshape(n, self.Hq, self.D)
                mag[r:r + n] = torch.einsum("hgnl,lhd->nhgd", w, v.abs()).reshape(n, self.Hq, self.D)
            r += n
        return out, mag
