"""GPU tests of the normed rotary queries and keys and their fused store against a 64-bit reference.

Tolerance: the result rounds to bf16 by at most 2^-8 of itself.  Before that, with y the normed head: the sum of at
most 256 squares errs by less than 2^-19 of itself in fp32 (16 in a row, then at most 16 more), its root by half of
that, and root, weights, products, cosine and sine by a few 2^-24 each: together at most 2^-18 (|y_i| + |y_j|) of the
pair's elements.
"""
import numpy as np
import pytest
import torch

from i8_reference import rope as rope64
from paged_kv_cache_62_gb300 import pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def freqs(rot, base=1.0e6):
    half = rot // 2
    return (base ** (-np.arange(half) / half)).astype(np.float32)


def inputs(T, Hq, Hkv, D, seed, wide=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = torch.exp(2 * torch.randn(T, Hq + 2 * Hkv, 1, generator=g, device="cuda"))  # heads of unequal size
    qkv = (torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda") * size).bfloat16().view(T, -1)
    q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:]
    parts = [t.view(T, -1, D) for t in (q, k, v)]
    w = [1 + 0.5 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    return (parts if wide else [t.contiguous() for t in parts]) + w


def close(got, x, w, eps, pos, inv, axis_of, inter, what):
    x = x.cpu().double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.cpu().double()
    want = rope64(y, pos, inv, axis_of, inter)
    # the pair's other element, where there is one
    pair = y.abs()
    half = len(inv)
    if inter:
        pair[..., 0:2 * half] = pair[..., 0:2 * half].unflatten(-1, (half, 2)).sum(-1, keepdim=True).expand(
            *pair.shape[:-1], half, 2).flatten(-2)
    else:
        pair[..., :2 * half] = (pair[..., :half] + pair[..., half:2 * half]).repeat(1, 1, 2)
    off = (got.cpu().double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -18 * pair)
    assert off.max() <= 0, f"{what}: over by {off.max():.3g}"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [(1, 16, 8, 128, 128), (37, 14, 2, 64, 64), (64, 4, 2, 64, 32),
                                            (5, 3, 1, 96, 48), (130, 32, 8, 128, 64), (3, 2, 2, 256, 256),
                                            (9, 1, 1, 16, 16), (17, 40, 40, 80, 80), (2, 5, 1, 208, 16),
                                            (4000, 16, 8, 128, 128), (700, 7, 3, 48, 32)])
def test_norm_rope(T, Hq, Hkv, D, rot, inter):
    q, k, _, qw, kw = inputs(T, Hq, Hkv, D, T + rot)
    inv, eps = freqs(rot), 1e-6
    pos = np.arange(T)[None] * 37 + 5
    qo, ko = (torch.full(t.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for t in (q, k))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.qk_norm_rope(q, k, qw, kw, eps, torch.tensor(pos[0], dtype=torch.int32, device="cuda"),
                     torch.from_numpy(inv).cuda(), qo, ko, interleaved=inter, err_word=err)
    assert err.item() == 0
    zero = np.zeros(rot // 2, int)
    close(qo, q, qw, eps, pos, inv, zero, inter, "q")
    close(ko, k, kw, eps, pos, inv, zero, inter, "k")


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("weights", ["both", "q", "none"])
def test_norm_rope_store(axes, inter, weights):
    T, Hq, Hkv, D, bs, NB = 200, 16, 8, 128, 16, 20
    rng = np.random.default_rng(axes)
    q, k, v, qw, kw = inputs(T, Hq, Hkv, D, axes)
    qw, kw = qw if weights != "none" else None, kw if weights == "both" else None
    inv, eps = freqs(D), 1e-3
    pos = rng.integers(0, 4000, (axes, T))
    axis_of = rng.integers(0, axes, D // 2)
    slots = rng.permutation(NB * bs)[:T]
    slots[3] = slots[77] = -1
    kc, vc = (torch.full((NB, bs, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    pkv.qk_norm_rope_store(q, k, v, qw, kw, eps, i32(pos), torch.from_numpy(inv).cuda(), i32(slots), qo, kc, vc,
                           freq_axis=i32(axis_of), interleaved=inter, err_word=err)
    assert err.item() == 0
    close(qo, q, qw, eps, pos, inv, axis_of, inter, "q")
    keep = torch.from_numpy(slots >= 0).cuda()
    at = torch.from_numpy(slots[slots >= 0].astype(np.int64)).cuda()
    close(kc.view(-1, Hkv, D)[at], k[keep], kw, eps, pos[:, slots >= 0], inv, axis_of, inter, "k")
    assert torch.equal(vc.view(-1, Hkv, D)[at], v[keep])
    rest = torch.ones(NB * bs, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.all(kc.view(-1, Hkv, D)[rest] == 7.0) and torch.all(vc.view(-1, Hkv, D)[rest] == 7.0)


def test_zeros_tiny_and_not_finite_heads():
    """A head of zeros stays zeros, tiny heads are ruled by eps, and a head with an infinity or NaN spoils itself only."""
    T, Hq, Hkv, D = 4, 3, 1, 64
    q, k, _, qw, kw = inputs(T, Hq, Hkv, D, 3, wide=False)
    q[0, 0] = 0
    q[1, 1] = 1e-20
    q[2, 2, 5], q[3, 0, 1] = float("inf"), float("nan")
    inv, pos = freqs(D), np.arange(T)[None]
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.qk_norm_rope(q, k, qw, kw, 1e-6, torch.arange(T, dtype=torch.int32, device="cuda"),
                     torch.from_numpy(inv).cuda(), qo, ko)
    assert not qo[0, 0].any()
    assert torch.isnan(qo[2, 2]).any() and torch.isnan(qo[3, 0]).any()
    ok = torch.ones(T, Hq, dtype=torch.bool)
    ok[2, 2] = ok[3, 0] = False
    for t in range(T):
        h = ok[t].nonzero()[:, 0].tolist()
        close(qo[t:t + 1, h], q[t:t + 1, h], qw, 1e-6, pos[:, t:t + 1], inv, np.zeros(D // 2, int), False, f"row {t}")


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D", [80, 128])
def test_norm_rope_in_place(inter, D):
    T, Hq, Hkv = 33, 8, 4
    q, k, _, qw, kw = inputs(T, Hq, Hkv, D, 1)
    inv, pos = torch.from_numpy(freqs(D)).cuda(), torch.arange(T, dtype=torch.int32, device="cuda")
    qo, ko = (torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k))
    pkv.qk_norm_rope(q, k, qw, kw, 1e-5, pos, inv, qo, ko, interleaved=inter)
    pkv.qk_norm_rope(q, k, qw, kw, 1e-5, pos, inv, q, k, interleaved=inter)
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_captured_store_replays_and_bad_slots_are_flagged():
    T, Hq, Hkv, D, bs, NB = 3, 16, 8, 128, 16, 4
    q, k, v, qw, kw = inputs(T, Hq, Hkv, D, 5, wide=False)
    inv = freqs(D)
    pos, slots = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
    slots.fill_(-1)
    kc, vc = (torch.zeros(NB, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo = torch.empty_like(q)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    invd = torch.from_numpy(inv).cuda()
    call = lambda: pkv.qk_norm_rope_store(q, k, v, qw, kw, 1e-6, pos, invd, slots, qo, kc, vc, err_word=err)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    zero = np.zeros(D // 2, int)
    for p, s, flag in (([0, 1, 2], [5, 6, 40], 0), ([9, 77, 3], [-1, 63, 64], pkv.ERR_SLOT_RANGE)):
        pos.copy_(torch.tensor(p, dtype=torch.int32))
        slots.copy_(torch.tensor(s, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert err.item() == flag
        close(qo, q, qw, 1e-6, np.array([p]), inv, zero, False, "q")
        at = [i for i in range(T) if 0 <= s[i] < NB * bs]
        rows = [s[i] for i in at]
        close(kc.view(-1, Hkv, D)[rows], k[at], kw, 1e-6, np.array([[p[i] for i in at]]), inv, zero, False, "k")
        assert torch.equal(vc.view(-1, Hkv, D)[rows], v[at])


def test_a_layer_of_a_windowed_model_over_an_int8_cache():
    """qk_norm_rope, kv_store_i8, paged_attention_window_i8 for prompts, then decode steps, then a drafted tree: as an
    engine runs them, against 64 bits over the same codes."""
    from mask_reference import random_trees, tree_sees, window_sees
    Hq, Hkv, D, bs, window, sinks = 8, 2, 64, 16, 40, 4
    prompts = [70, 5, 33]
    B, mb = len(prompts), 16
    bt = torch.arange(B * mb, dtype=torch.int32, device="cuda").view(B, mb)
    kc, vc, sc = pkv.alloc_i8_cache(B * mb, bs, Hkv, D)
    inv = torch.from_numpy(freqs(D)).cuda()
    lens = [0] * B
    ws = pkv.alloc_attention_workspace(sum(prompts) + 100, Hq, Hkv, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    steps = [(prompts, "window"), ([1] * B, "decode"), ([1] * B, "decode"), ([9] * B, "tree"), ([1] * B, "decode")]
    for step, (new, kind) in enumerate(steps):
        lens = [a + n for a, n in zip(lens, new)]
        T = sum(new)
        q, k, v, qw, kw = inputs(T, Hq, Hkv, D, step)
        v.clamp_(-4, 4)
        pos = i32(np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)]))
        pkv.qk_norm_rope(q, k, qw, kw, 1e-6, pos, inv, q, k, err_word=err)
        cu, ld = i32(np.concatenate([[0], np.cumsum(new)])), i32(lens)
        pkv.kv_store_i8(k, v, kc, vc, sc, bt, ld, cu, err_word=err)
        qd = q.contiguous()
        out = torch.empty_like(qd)
        if kind == "decode":
            pkv.paged_decode_window_i8(qd, kc, vc, sc, bt, ld, D ** -0.5, window, sinks, out, ws, err_word=err)
            sees = [window_sees(L, 1, window, sinks) for L in lens]
        elif kind == "window":
            pkv.paged_attention_window_i8(qd, kc, vc, sc, bt, cu, ld, D ** -0.5, window, sinks, out, ws, err_word=err)
            sees = [window_sees(L, n, window, sinks) for L, n in zip(lens, new)]
        else:
            masks = random_trees(new, 1, np.random.default_rng(0))
            pkv.paged_attention_tree_i8(qd, kc, vc, sc, bt, None, ld, torch.from_numpy(masks).cuda(), D ** -0.5, out, ws,
                                        err_word=err, new_per_seq=9)
            sees = [tree_sees(L, 9, masks[9 * b:9 * b + 9]) for b, L in enumerate(lens)]
        assert err.item() == 0
        wide = sc.double().repeat_interleave(16, 1)
        kd, vd = kc.double() * wide[..., 0:1], vc.double() * wide[..., 1:2]
        r = 0
        for b, s in enumerate(sees):
            n, L = s.shape
            rows = lambda c: c[bt[b].long()].reshape(-1, Hkv, D)[:L]
            x = torch.einsum("nhgd,lhd->hgnl", qd[r:r + n].double().view(n, Hkv, -1, D), rows(kd)) * D ** -0.5
            w = torch.softmax(x.masked_fill(~torch.from_numpy(s).cuda(), float("-inf")), -1)
            want = torch.einsum("hgnl,lhd->nhgd", w, rows(vd)).reshape(n, Hq, D)
            mag = torch.einsum("hgnl,lhd->nhgd", w, rows(vd).abs()).reshape(n, Hq, D)
            # int8 caches: weights 2^-11, scores 2^-12 at magnitudes below 2^6 (see test_gpu_i8.py)
            off = (out[r:r + n].double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -10 * mag)
            assert off.max() <= 0, (step, kind, off.max().item())
            r += n


def test_a_layer_over_a_bf16_cache():
    """qk_norm_rope_store, then windowed prompts, decode steps and a drafted tree over one bf16 cache and workspace."""
    from mask_reference import random_trees, tree_sees, window_sees
    Hq, Hkv, D, bs, window, sinks = 8, 2, 128, 32, 100, 3
    prompts = [700, 1, 140, 64]
    B, mb = len(prompts), 24
    bt = torch.randperm(B * mb, generator=torch.Generator().manual_seed(1)).int().cuda().view(B, mb)
    kc, vc = (torch.full((B * mb, bs, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    inv = torch.from_numpy(freqs(D)).cuda()
    lens = [0] * B
    ws = pkv.alloc_attention_workspace(sum(prompts), Hq, Hkv, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    for step, (new, kind) in enumerate([(prompts, "window"), ([1] * B, "decode"), ([20] * B, "tree"), ([1] * B, "decode"),
                                        ([3, 0, 1, 7], "window"), ([4] * B, "tree")]):
        lens = [a + n for a, n in zip(lens, new)]
        T = sum(new)
        q, k, v, qw, kw = inputs(T, Hq, Hkv, D, step)
        v.clamp_(-4, 4)
        pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)])
        seq = np.repeat(np.arange(B), new)
        slots = bt.cpu().numpy()[seq, pos // bs].astype(np.int64) * bs + pos % bs
        qd = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        pkv.qk_norm_rope_store(q, k, v, qw, kw, 1e-6, i32(pos), inv, i32(slots), qd, kc, vc, err_word=err)
        cu, ld = i32(np.concatenate([[0], np.cumsum(new)])), i32(lens)
        out = torch.full_like(qd, float("nan"))
        if kind == "decode":
            pkv.paged_decode_window(qd, kc, vc, bt, ld, D ** -0.5, window, sinks, out, ws, err_word=err)
        elif kind == "window":
            pkv.paged_attention_window(qd, kc, vc, bt, cu, ld, D ** -0.5, window, sinks, out, ws, err_word=err)
        if kind != "tree":
            sees = [window_sees(L, n, window, sinks) for L, n in zip(lens, new)]
        else:
            masks = random_trees(new, 1, np.random.default_rng(step))
            pkv.paged_attention_tree(qd, kc, vc, bt, None, ld, torch.from_numpy(masks).cuda(), D ** -0.5, out, ws,
                                     err_word=err, new_per_seq=new[0])
            sees = [tree_sees(L, n, masks[n * b:n * b + n]) for b, (L, n) in enumerate(zip(lens, new))]
        assert err.item() == 0
        r = 0
        for b, s in enumerate(sees):
            n, L = s.shape
            rows = lambda c: c[bt[b].long()].reshape(-1, Hkv, D)[:L].double()
            x = torch.einsum("nhgd,lhd->hgnl", qd[r:r + n].double().view(n, Hkv, Hq // Hkv, D), rows(kc)) * D ** -0.5
            w = torch.softmax(x.masked_fill(~torch.from_numpy(s).cuda(), float("-inf")), -1)
            want = torch.einsum("hgnl,lhd->nhgd", w, rows(vc)).reshape(n, Hq, D)
            mag = torch.einsum("hgnl,lhd->nhgd", w, rows(vc).abs()).reshape(n, Hq, D)
            # bf16 caches: weights 2^-8 on the tile, scores 2^-12 at magnitudes below 2^6 (see test_gpu_masks.py)
            off = (out[r:r + n].double() - want).abs() - (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11) * mag)
            assert n == 0 or off.max() <= 0, (step, kind, off.max().item())
            r += n
