"""Measured cases of normed rotary queries and keys, of attention through a sliding window with sinks, and of
attention for trees of drafted tokens.

Three operators a serving engine runs over its paged KV cache, each with a plain form (elementary torch
operations) and, with ``own`` set, the library's calls:

* ``norm``   -- root-mean-square norm of every query and key head with a learned weight, and rotary positions
  (one axis or several) in the same pass; k and v stored through slots, or q and k returned;
* ``window`` -- attention that sees the last ``window`` keys of a sequence and its first ``sinks``: one new
  token a sequence (``new`` "one") or several, over bf16 and int8 caches.  Pages no query sees are not held:
  their table entries are -1;
* ``tree``   -- attention of a sequence's drafted tokens, stored at its last positions: each sees the
  sequence before the draft, and of the draft the nodes in its bit mask (its ancestors and itself).

Head layouts, page sizes and lengths are those of the package's workloads (16 q / 8 kv heads of 128, pages of
256; 14 / 2 heads of 64, pages of 16; the tiny batch; the long/mixed batch).
"""
from __future__ import annotations

import math
import zlib

import numpy as np
import torch

own = False

SB = 16  # tokens that share a scale in an int8 cache (per kv head, one for K and one for V)
EPS = 1e-6


# ------------------------------------------------------------------------------------------ the cases
def listed():
    big = dict(Hq=16, Hkv=8, D=128, bs=256)
    return [
        # a decode step's q and k of 64 sequences, k and v stored: the latency of one call a layer and step
        dict(name="norm_step", op="norm", T=64, rot=128, axes=1, pairs="halves", far=4096, store=True, **big),
        # a long prompt
        dict(name="norm_prompt", op="norm", T=16384, rot=128, axes=1, pairs="halves", far=32768, store=True, **big),
        # images and video among text, a part of each head turned, q and k kept (for a cache of another type)
        dict(name="norm_video", op="norm", T=1531, Hq=14, Hkv=2, D=80, bs=16, rot=48, axes=3, pairs="adjacent",
             far=1 << 20, store=False),
        # four short sequences: the smallest call, all latency
        dict(name="window_tiny", op="window", cache="bf16", B=4, Hq=4, Hkv=2, D=64, bs=16, lo=1, hi=400,
             dist="uniform", window=128, sinks=4, new="one"),
        # the ordinary decode step
        dict(name="window_step", op="window", cache="bf16", B=64, lo=512, hi=4096, dist="uniform", window=1024, sinks=4,
             new="one", **big),
        # long and short sequences together, small pages: the largest read
        dict(name="window_long_mixed", op="window", cache="bf16", B=256, Hq=16, Hkv=8, D=128, bs=16, lo=1, hi=32768,
             dist="log", window=4096, sinks=64, new="one"),
        # the same model over an int8 cache, all sequences longer than the window
        dict(name="window_int8", op="window", cache="int8", B=96, Hq=16, Hkv=8, D=128, bs=64, lo=4096, hi=32768,
             dist="log", window=2048, sinks=16, new="one"),
        # a 64-token chunk of prefill a sequence over a cached prefix
        dict(name="window_chunk64", op="window", cache="bf16", B=64, lo=512, hi=4096, dist="uniform", window=1024,
             sinks=4, new=64, **big),
        # whole prompts of ragged lengths, some far longer than the window
        dict(name="window_prompts", op="window", cache="bf16", B=7, lo=1, hi=2048, dist="uniform", window=512, sinks=1,
             new="all", **big),
        # a few drafted tokens of four short sequences: all latency
        dict(name="tree_tiny", op="tree", cache="bf16", B=4, Hq=4, Hkv=2, D=64, bs=16, lo=8, hi=100, dist="uniform",
             new=7),
        # the verify step of 32-node trees
        dict(name="tree_step", op="tree", cache="bf16", B=64, lo=512, hi=4096, dist="uniform", new=32, **big),
        # trees of any size over an int8 cache, 7 query heads a kv head
        dict(name="tree_ragged_int8", op="tree", cache="int8", B=48, Hq=14, Hkv=2, D=64, bs=16, lo=100, hi=4096,
             dist="log", new="ragged"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# bytes and operations of the largest listed case of each operator bound the drawn ones
_MOST = {"norm": (270e6, 1e12), "window": (1.5e9, 5.0e10), "tree": (650e6, 7.5e10)}


def draw(rng):
    case = _draw(rng)
    while True:
        w, most = work(case), _MOST[case["op"]]
        rows = 0 if case["op"] == "norm" else int(_lengths(case, 0)[1].sum())
        if w["bytes"] <= most[0] and w["flops"] <= most[1] and rows <= 6000:
            return case
        for key in ("T", "B"):  # fewer rows or sequences
            if case.get(key, 1) > 1:
                case[key] //= 2
                break
        else:
            case["hi"] = max(case["lo"], case["hi"] // 2)
            case["lo"] = max(1, case["lo"] // 2)


def _draw(rng):
    op = rng.choice(["norm", "window", "window", "tree"])
    Hq, Hkv = rng.choice([(4, 2), (14, 2), (16, 8), (16, 16), (32, 8), (8, 1), (12, 4), (6, 3), (16, 1), (15, 5)])
    bs = rng.choice([16, 32, 64, 128, 256, 512])
    if op == "norm":
        D = rng.choice([64, 80, 96, 128, 256])
        return dict(op=op, T=_log(rng, 1, 16384), Hq=Hq, Hkv=Hkv, D=D, bs=bs, rot=rng.choice([D, D // 32 * 16, 32]),
                    axes=rng.choice([1, 2, 3]), pairs=rng.choice(["halves", "adjacent"]), far=_log(rng, 2, 1 << 20),
                    store=rng.random() < 0.6)
    case = dict(op=op, cache=rng.choice(["bf16", "bf16", "int8"]), B=_log(rng, 1, 256), Hq=Hq, Hkv=Hkv,
                D=rng.choice([64, 128]), bs=bs, dist=rng.choice(["uniform", "log"]))
    if op == "window":
        new = rng.choice(["one", "one", 2, 5, 16, 64, "ragged", "all"])
        hi = _log(rng, 2, 32768 if new == "one" else 4096)
        case.update(window=_log(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 16, rng.randint(1, 300)]))
    else:
        new = rng.choice([1, 3, 7, 8, 13, 16, 25, 32, 64, "ragged"])
        hi = _log(rng, 2, 4096)
    least = new if not isinstance(new, str) else 1
    hi = max(hi, least)
    case.update(lo=rng.randint(least, hi), hi=hi, new=new)
    return case


# ------------------------------------------------------------------------------------------ inputs
def _lengths(case, seed):
    """Context lengths (new tokens counted) and the new tokens of every sequence: those of the case, so that
    every seed's tensors have the same shapes, in the seed's order; and the seed's generator."""
    rng = np.random.default_rng(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if case["dist"] == "log":
        L = np.exp(rng.uniform(math.log(lo), math.log(hi + 1), B)).astype(np.int64).clip(lo, hi)
    else:
        L = rng.integers(lo, hi, B, endpoint=True)
    new = case["new"]
    if new == "one":
        n = np.ones(B, np.int64)
    elif new == "all":
        n = L.copy()
    elif new == "ragged":  # single tokens and chunks of up to 512, trees of up to 100 nodes
        n = np.exp(rng.uniform(0, math.log(100 if case["op"] == "tree" else 512), B)).astype(np.int64)
        n[rng.random(B) < 0.2] = 1
        n = np.minimum(n, L)
    else:
        n = np.full(B, new, np.int64)
    rng = np.random.default_rng(seed)
    order = rng.permutation(B)
    return L[order], n[order], rng


def _seen(case, L, n):
    """Half-open ranges of the positions that some query of a sequence sees."""
    if case["op"] == "tree":
        return [(0, L)]
    head = min(case["sinks"], L)
    tail = max(head, L - n - case["window"] + 1)
    return [(0, head), (tail, L)]


def _tables(case, L, n, rng, extra=3):
    bs = case["bs"]
    held = []
    for l, m in zip(L, n):
        pages = set()
        for a, b in _seen(case, int(l), int(m)):
            pages.update(range(a // bs, -(-b // bs)) if b > a else ())
        held.append(sorted(pages))
    NB = sum(map(len, held)) + extra
    perm = rng.permutation(NB)
    bt = np.full((len(L), int(-(-L.max() // bs))), -1, np.int64)
    cur = 0
    for b, pages in enumerate(held):
        bt[b, pages] = perm[cur:cur + len(pages)]
        cur += len(pages)
    return bt, NB


def _filled(bt, L, bs, NB):
    filled = np.zeros(NB, np.int64)
    for b in range(len(L)):
        pages = np.nonzero(bt[b] >= 0)[0]
        filled[bt[b, pages]] = np.clip(L[b] - pages * bs, 0, bs)
    return filled


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda").bfloat16()


def _pool(case, NB, filled, gen):
    """A cache whose first `filled[p]` rows of page p hold values: K with channels of unequal size, V without.
    The other rows hold what an earlier owner left: NaN, or codes whose scales are NaN."""
    dev = torch.device("cuda")
    bs, Hkv, D = case["bs"], case["Hkv"], case["D"]
    chan = torch.exp(0.5 * torch.randn(Hkv, D, generator=gen, device=dev))
    live = torch.arange(bs, device=dev).view(1, bs) < torch.as_tensor(filled, device=dev).view(NB, 1)
    step = max(1, (64 << 20) // (bs * Hkv * D))
    if case["cache"] == "bf16":
        kc = torch.empty(NB, bs, Hkv, D, dtype=torch.bfloat16, device=dev)
        vc = torch.empty_like(kc)
        for p in range(0, NB, step):
            m = live[p:p + step, :, None, None]
            for which, c in ((0, kc), (1, vc)):
                x = torch.randn(m.shape[0], bs, Hkv, D, generator=gen, device=dev)
                c[p:p + step] = torch.where(m, x * chan if which == 0 else x, float("nan")).bfloat16()
        return kc, vc, None
    kc = torch.empty(NB, bs, Hkv, D, dtype=torch.int8, device=dev)
    vc = torch.empty_like(kc)
    sc = torch.empty(NB, bs // SB, Hkv, 2, dtype=torch.float32, device=dev)
    for p in range(0, NB, step):
        m = live[p:p + step].view(-1, bs // SB, SB, 1, 1)
        for which, c in ((0, kc), (1, vc)):
            x = torch.randn(m.shape[0], bs // SB, SB, Hkv, D, generator=gen, device=dev)
            if which == 0:
                x *= chan
            s = (x * m).abs().amax(dim=(2, 4)) / 127
            c[p:p + step] = torch.round(x / s.clamp_min(1e-3).view(-1, bs // SB, 1, Hkv, 1)).clamp(-127, 127).to(
                torch.int8).view(-1, bs, Hkv, D)
            sc[p:p + step, :, :, which] = torch.where(m.any(dim=2).view(-1, bs // SB, 1), s, float("nan"))
    return kc, vc, sc


def _trees(n, rng):
    """Bit masks of random trees, int32 [rows, words]: bit j of row i is set if node j is an ancestor of node i
    or i itself.  A sequence's node 0 is the root; a later node's parent is one of the eight before it."""
    words = -(-int(n.max()) // 32)
    masks = []
    for m in n.tolist():
        sees = np.zeros((m, 32 * words), np.uint8)
        for i in range(m):
            if i:
                sees[i] = sees[i - 1 - int(rng.integers(0, min(i, 8)))]
            sees[i, i] = 1
        masks.append(np.packbits(sees, axis=1, bitorder="little"))
    return np.ascontiguousarray(np.concatenate(masks)).view(np.int32).reshape(-1, words)


def _inputs(case, seed):
    """The tensors of a case, from its seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
    i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=dev)
    if case["op"] == "norm":
        rng = np.random.default_rng(seed)
        T, rot, axes = case["T"], case["rot"], case["axes"]
        # q, k and v are the parts of one projection's rows, whose channels and tokens differ in size
        size = torch.exp(torch.randn((Hq + 2 * Hkv) * D, generator=gen, device=dev))
        qkv = (torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device=dev) * size
               * torch.exp(torch.randn(T, 1, generator=gen, device=dev))).bfloat16()
        qw, kw = ((1 + 0.3 * torch.randn(D, generator=gen, device=dev)).bfloat16().float() for _ in range(2))
        half = rot // 2
        inv = torch.as_tensor((1.0e6 ** (-np.arange(half) / half)).astype(np.float32), device=dev)
        # a quarter of the frequencies for the first axis (time), the rest in equal parts, in order
        bound = [0, half] if axes == 1 else [0, half // 4] + [half // 4 + (half - half // 4) * a // (axes - 1)
                                                              for a in range(1, axes)]
        axis_of = np.zeros(half, np.int32)
        for a in range(axes):
            axis_of[bound[a]:bound[a + 1]] = a
        # text runs on all axes together; an image spreads over rows and columns at one time
        start = int(rng.integers(0, case["far"]))
        pos = np.tile(start + np.arange(T), (axes, 1))
        if axes > 1:
            side = int(rng.integers(2, 40))
            t = np.arange(T)
            frame = (t // (side * side)) % 2 == 1
            pos[0, frame] = start + (t[frame] // (side * side)) * side * side
            pos[1, frame] = pos[0, frame] + (t[frame] // side) % side
            pos[axes - 1, frame] = pos[0, frame] + t[frame] % side
        q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:]
        d = dict(q=q.view(T, Hq, D), k=k.view(T, Hkv, D), v=v.view(T, Hkv, D), qw=qw, kw=kw, pos=i32(pos), inv=inv,
                 axis_of=i32(axis_of), q_out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev))
        if case["store"]:
            NB = -(-T // bs) + 2
            slots = (rng.permutation(NB)[:, None] * bs + np.arange(bs)[None]).reshape(-1)[:T]
            slots[rng.random(T) < 0.01] = -1  # rows whose K/V is cached already
            d["kc"], d["vc"] = (torch.zeros(NB, bs, Hkv, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
            d["slots"] = i32(slots)
        else:
            d["k_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev)
        return d
    L, n, rng = _lengths(case, seed)
    bt, NB = _tables(case, L, n, rng)
    kc, vc, sc = _pool(case, NB, _filled(bt, L, bs, NB), gen)
    T = int(n.sum())
    d = dict(kc=kc, vc=vc, sc=sc, bt=i32(bt), lens=i32(L), cu=i32(np.concatenate([[0], np.cumsum(n)])), L=L.tolist(),
             n=n.tolist(), max_len=int(L.max()), q=_randn(gen, T, Hq, D),
             out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev), scale=1.0 / math.sqrt(D))
    if case["op"] == "tree":
        d["mask"] = i32(_trees(n, rng))
    return d


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] != "norm":
            from paged_kv_cache_62_gb300 import pkv
            T, Hq, D = st["q"].shape
            alloc = pkv.alloc_workspace if case["new"] == "one" else pkv.alloc_attention_workspace
            st["ws"] = alloc(T, Hq, case["Hkv"], D)
    return st


# ------------------------------------------------------------------------------------------ one pass
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from paged_kv_cache_62_gb300 import pkv
    case = st["case"]
    if case["op"] == "norm":
        how = dict(freq_axis=st["axis_of"], interleaved=case["pairs"] == "adjacent", err_word=st["err"])
        if case["store"]:
            pkv.qk_norm_rope_store(st["q"], st["k"], st["v"], st["qw"], st["kw"], EPS, st["pos"], st["inv"], st["slots"],
                                   st["q_out"], st["kc"], st["vc"], **how)
            return st["q_out"], st["kc"], st["vc"]
        pkv.qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], EPS, st["pos"], st["inv"], st["q_out"], st["k_out"], **how)
        return st["q_out"], st["k_out"]
    int8 = case["cache"] == "int8"
    cache = (st["kc"], st["vc"], st["sc"]) if int8 else (st["kc"], st["vc"])
    how = dict(max_context_len=st["max_len"], err_word=st["err"])
    if case["new"] == "one":
        call = pkv.paged_decode_window_i8 if int8 else pkv.paged_decode_window
        call(st["q"], *cache, st["bt"], st["lens"], st["scale"], case["window"], case["sinks"], st["out"], st["ws"],
             **how)
        return st["out"]
    n = 0 if isinstance(case["new"], str) else case["new"]
    cu = None if n else st["cu"]
    if case["op"] == "window":
        call = pkv.paged_attention_window_i8 if int8 else pkv.paged_attention_window
        call(st["q"], *cache, st["bt"], cu, st["lens"], st["scale"], case["window"], case["sinks"], st["out"], st["ws"],
             new_per_seq=n, **how)
    else:
        call = pkv.paged_attention_tree_i8 if int8 else pkv.paged_attention_tree
        call(st["q"], *cache, st["bt"], cu, st["lens"], st["mask"], st["scale"], st["out"], st["ws"], new_per_seq=n,
             **how)
    return st["out"]


def _run_plain(st):
    return _plain_norm(st) if st["case"]["op"] == "norm" else _plain_attend(st)


def _plain_norm(st):
    case = st["case"]
    rot, half = case["rot"], case["rot"] // 2
    # angles in 64 bits: a far position times a frequency keeps few of 32 bits after its whole turns
    ang = st["pos"].double()[st["axis_of"].long()] * st["inv"].double()[:, None]      # [half, T]
    cos, sin = ang.cos().float().t()[:, None], ang.sin().float().t()[:, None]          # [T, 1, half]

    def turn(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        if case["pairs"] == "halves":
            a, b = x[..., :half], x[..., half:rot]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([r, x[..., rot:]], -1).bfloat16()

    st["q_out"].copy_(turn(st["q"], st["qw"]))
    if not case["store"]:
        st["k_out"].copy_(turn(st["k"], st["kw"]))
        return st["q_out"], st["k_out"]
    keep = (st["slots"] >= 0).nonzero()[:, 0]
    at = st["slots"][keep].long()
    for cache, new in ((st["kc"], turn(st["k"], st["kw"])), (st["vc"], st["v"])):
        cache.view(-1, *cache.shape[2:])[at] = new[keep]
    return st["q_out"], st["kc"], st["vc"]


def _rows(st, b):
    """Positions of sequence b that some query sees, and their K and V rows in fp32 [Hkv, positions, D]."""
    case = st["case"]
    bs, Hkv, D = case["bs"], case["Hkv"], case["D"]
    dev = st["kc"].device
    pos = torch.cat([torch.arange(x, y, device=dev) for x, y in _seen(case, st["L"][b], st["n"][b])])
    slot = st["bt"][b].long()[pos // bs] * bs + pos % bs
    k, v = (c.view(-1, Hkv, D)[slot].float() for c in (st["kc"], st["vc"]))
    if case["cache"] == "int8":
        s = st["sc"].view(-1, Hkv, 2)[slot // SB]
        k, v = k * s[..., 0:1], v * s[..., 1:2]
    return pos, k.permute(1, 0, 2), v.permute(1, 0, 2)


def _plain_attend(st):
    case = st["case"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G, r = Hq // Hkv, 0
    for b, (L, n) in enumerate(zip(st["L"], st["n"])):
        pos, k, v = _rows(st, b)
        q = st["q"][r:r + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
        s = torch.matmul(q, k.transpose(1, 2)) * st["scale"]
        if case["op"] == "tree":
            node = pos - (L - n)
            word, bit = (node.clamp_min(0) // 32), (node % 32)
            seen = (node < 0) | ((st["mask"][r:r + n].long()[:, word] >> bit) & 1 == 1)
        else:
            at = (L - n + torch.arange(n, device=s.device))[:, None]
            seen = (pos <= at) & ((pos > at - case["window"]) | (pos < case["sinks"]))
        s = s.view(Hkv, G, n, -1).masked_fill(~seen, float("-inf")).view(Hkv, G * n, -1)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        st["out"][r:r + n] = o.view(Hkv, G, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D).bfloat16()
        r += n
    return st["out"]


# ------------------------------------------------------------------------------------------ in 64 bits
def _exact_norm(case, st):
    f64 = torch.float64
    rot, half, Hkv, D = case["rot"], case["rot"] // 2, case["Hkv"], case["D"]
    turns = torch.zeros(case["T"], half, dtype=f64, device="cuda")
    for i, a in enumerate(st["axis_of"].tolist()):
        turns[:, i] = st["pos"][a].to(f64) * float(st["inv"][i])
    z = torch.polar(torch.ones_like(turns), turns)
    first, second = ((slice(0, half), slice(half, rot)) if case["pairs"] == "halves"
                     else (slice(0, rot, 2), slice(1, rot, 2)))

    def turn(x, w):
        y = x.to(f64)
        y = y / (torch.linalg.vector_norm(y, dim=-1, keepdim=True).square() / D + EPS).sqrt() * w.to(f64)
        t = torch.complex(y[..., first], y[..., second]) * z[:, None]
        y[..., first], y[..., second] = t.real, t.imag
        return y

    if not case["store"]:
        return turn(st["q"], st["qw"]), turn(st["k"], st["kw"])
    kc, vc = (torch.zeros(c.shape, dtype=f64, device="cuda") for c in (st["kc"], st["vc"]))
    keep = st["slots"] >= 0
    at = st["slots"][keep].long()
    kc.view(-1, Hkv, D)[at] = turn(st["k"], st["kw"])[keep]
    vc.view(-1, Hkv, D)[at] = st["v"][keep].to(f64)
    return turn(st["q"], st["qw"]), kc, vc


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, st)
    f64 = torch.float64
    Hkv, D, bs = case["Hkv"], case["D"], case["bs"]
    G = case["Hq"] // Hkv
    if work(case)["flops"] > 3e11:
        return None
    out, r = torch.empty(st["q"].shape, dtype=f64, device="cuda"), 0
    for b, (L, n) in enumerate(zip(st["L"], st["n"])):
        # what each query sees, over all positions; then the columns that anyone sees
        sees = np.zeros((n, L), bool)
        if case["op"] == "tree":
            sees[:, :L - n] = True
            bits = np.unpackbits(st["mask"][r:r + n].cpu().numpy().view(np.uint8), axis=1, bitorder="little")
            sees[:, L - n:] = bits[:, :n]
        else:
            for i in range(n):
                p = L - n + i
                sees[i, max(0, p + 1 - case["window"]):p + 1] = True
                sees[i, :min(case["sinks"], p + 1)] = True
        cols = np.nonzero(sees.any(0))[0]
        at = torch.as_tensor(cols, device="cuda")
        hide = ~torch.as_tensor(sees[:, cols], device="cuda")
        page, row = st["bt"][b].long()[at // bs], at % bs
        for h in range(Hkv):
            k, v = st["kc"][page, row, h].to(f64), st["vc"][page, row, h].to(f64)
            if case["cache"] == "int8":
                sc = st["sc"][page, row // SB].to(f64)
                k, v = k * sc[:, h, 0:1], v * sc[:, h, 1:2]
            x = torch.einsum("igd,jd->gij", st["q"][r:r + n, h * G:(h + 1) * G].to(f64), k) * st["scale"]
            x = torch.where(hide, -math.inf, x)
            out[r:r + n, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", torch.softmax(x, -1), v)
        r += n
    return out


# ------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
    if case["op"] == "norm":
        T, H = case["T"], Hq + (2 if case["store"] else 1) * Hkv
        return {"bytes": 4 * T * H * D + 4 * T * (case["axes"] + (1 if case["store"] else 0)) + 8 * D,
                "flops": T * (Hq + Hkv) * (4 * D + 3 * case["rot"])}
    L, n, rng = _lengths(case, 0)
    T = int(n.sum())
    seen = pairs = pages = blocks = 0
    for l, m in zip(L.tolist(), n.tolist()):
        for a, b in _seen(case, l, m):
            if b > a:
                seen += b - a
                pages += -(-b // bs) - a // bs
                blocks += -(-b // SB) - a // SB
        if case["op"] == "tree":  # the mask says which of the nodes; a node counts half the earlier ones
            pairs += m * (l - m) + m * (m + 1) // 2
        else:
            p = np.arange(l - m, l)
            head = np.minimum(case["sinks"], p + 1)
            pairs += int((head + np.maximum(0, p + 1 - np.maximum(head, p + 1 - case["window"]))).sum())
    cached = seen * Hkv * 2 * D * (1 if case["cache"] == "int8" else 2) + (
        blocks * Hkv * 8 if case["cache"] == "int8" else 0)
    masks = 4 * T * (-(-int(n.max()) // 32)) if case["op"] == "tree" else 0
    return {"bytes": cached + 4 * T * Hq * D + 4 * pages + 8 * len(L) + masks, "flops": 4.0 * pairs * Hq * D}
