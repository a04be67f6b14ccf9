"""64-bit references of the int8 cache, the rotary positions and attention over dequantised rows (test
infrastructure: numpy and torch on the CPU, no library code)."""
import numpy as np
import torch

SB = 16


def rne(x):
    return np.rint(x)  # ties to even


def store_i8(k, v, kc, vc, sc, bt, lens, new):
    """In place on numpy arrays: k, v [T, Hkv, D] float64, codes int8 [NB, bs, Hkv, D], scales float32
    [NB, bs / 16, Hkv, 2]; new[b] rows of sequence b end at position lens[b]."""
    bs = kc.shape[1]
    r = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        p = L - n
        while p < L:
            base = p - p % SB
            end = min(L, base + SB)
            page, off = bt[b][base // bs], base % bs
            for which, x, c in ((0, k, kc), (1, v, vc)):
                rows = x[r:r + end - p]
                for h in range(kc.shape[2]):
                    a = np.abs(rows[:, h]).max()
                    s = np.float32(a) * (np.float32(1.0) / np.float32(127.0)) if np.isfinite(a) else np.float32("nan")
                    old = sc[page, off // SB, h, which]
                    if p > base:
                        s = np.float32("nan") if np.isnan(old) or np.isnan(s) else max(old, s)
                        if s > old:
                            kept = c[page, off:off + p - base, h].astype(np.float64) * np.float64(old)
                            c[page, off:off + p - base, h] = rne(kept / np.float64(s)).astype(np.int8)
                    if s > 0:
                        q = np.clip(rne(rows[:, h] / np.float64(s)), -127, 127).astype(np.int8)
                    else:
                        q = np.zeros(rows[:, h].shape, np.int8)
                    c[page, off + p - base:off + end - base, h] = q
                    sc[page, off // SB, h, which] = s
            r += end - p
            p = end


def attend_i8(q, kc, vc, sc, bt, lens, new, scale):
    """(out, mean): float64 [T, Hq, D], causal attention of each sequence's last n tokens, and the weighted mean
    of |v| that bounds the weights' rounding."""
    T, Hq, D = q.shape
    bs, Hkv = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    out, mag = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    r = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        if L > 0:
            pages = torch.as_tensor(bt[b][: -(-L // bs)].astype(np.int64))
            s = sc[pages].double().repeat_interleave(SB, 1).reshape(-1, Hkv, 2)[:L]
            kd = kc[pages].reshape(-1, Hkv, D)[:L].double() * s[..., 0:1]
            vd = vc[pages].reshape(-1, Hkv, D)[:L].double() * s[..., 1:2]
            for i in range(n):
                e = L - n + i + 1
                x = torch.einsum("hgd,lhd->hgl", q[r + i].double().view(Hkv, G, D), kd[:e]) * scale
                w = torch.softmax(x, -1)
                out[r + i] = torch.einsum("hgl,lhd->hgd", w, vd[:e]).reshape(Hq, D)
                mag[r + i] = torch.einsum("hgl,lhd->hgd", w, vd[:e].abs()).reshape(Hq, D)
        r += n
    return out, mag


def rope(x, pos, inv_freq, axis_of, interleaved):
    """float64 [T, H, D] of x turned: pos [axes, T] ints, inv_freq float32 [rot / 2]."""
    x = x.double().clone()
    half = len(inv_freq)
    p = np.asarray(pos, np.int64)[np.asarray(axis_of)].T                # [T, half]
    ang = p.astype(np.longdouble) * np.asarray(inv_freq, np.float32).astype(np.longdouble)
    ang = np.remainder(ang, 2 * np.longdouble("3.14159265358979323846264338327950288")).astype(np.float64)
    cos, sin = (torch.from_numpy(f(ang))[:, None] for f in (np.cos, np.sin))
    i, j = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half)))
    a, b = x[..., i].clone(), x[..., j].clone()
    x[..., i], x[..., j] = a * cos - b * sin, b * cos + a * sin
    return x
