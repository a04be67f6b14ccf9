"""GPU tests of attention through a sliding window with sinks and of trees of drafted tokens, over bf16, E4M3 and int8
caches.

Attention must stay within  2^-8 |out| + w A  of the 64-bit result, A = the softmax-weighted mean of |v|: the bf16
output rounds by at most 2^-8 of itself, and the weights' errors move it by at most their relative size times A.
bf16 caches: a weight is two bf16 parts (2^-16), its fp32 score errs by less than 2^-12 (scores stay below 2^6, a sum
of at most 128 products errs by less than 2^-14 of that), sums and merges have the rest of w = 2^-11.  Calls with
offsets, or with more new tokens a sequence than 16 / (query heads a kv head), run on the tensor-memory tile, which
rounds a weight to one bf16 part, 2^-8: w = 2^-8 + 2^-11 (long_runs).  E4M3 and int8
caches round it to f16, 2^-11, and their scores err by up to twice 2^-12: w = 2^-10.
"""
import numpy as np
import pytest
import torch

from mask_reference import Problem, random_trees, tree_sees, window_sees
from paged_kv_cache_62_gb300 import pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def check(out, prob, what, long_runs=False):
    want, mag = prob.want()
    got = out.cpu().double()
    assert torch.isfinite(got).all(), what
    w = 2.0 ** -10 if prob.cache != "bf16" else 2.0 ** -11 + (2.0 ** -8 if long_runs else 0.0)
    off = (got - want).abs() - (2.0 ** -8 * want.abs() + w * mag)
    assert off.max() <= 0, f"{what}: over the bound by {off.max():.3g}"


DECODE = {"bf16": "paged_decode_window", "fp8": "paged_decode_window_fp8", "int8": "paged_decode_window_i8"}


def decode(prob, window, sinks, workers=0, ws=None, dev=None, **kw):
    q, cache, bt, lens, _ = dev or prob.cuda()
    out = torch.full_like(q, float("nan"))
    ws = pkv.alloc_workspace(q.shape[0], prob.Hq, prob.Hkv, prob.D) if ws is None else ws
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    getattr(pkv, DECODE[prob.cache])(q, *cache, bt, lens, prob.scale, window, sinks, out, ws, num_workers=workers,
                                     err_word=err, **kw)
    assert err.item() == 0
    return out


def attend(prob, args, kind="window", uniform=0, workers=0, ws=None, err_is=0, dev=None):
    q, cache, bt, lens, cu = dev or prob.cuda()
    out = torch.full_like(q, float("nan"))
    ws = pkv.alloc_attention_workspace(q.shape[0], prob.Hq, prob.Hkv, prob.D) if ws is None else ws
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    fn = getattr(pkv, f"paged_attention_{kind}" + ("_i8" if prob.cache == "int8" else ""))
    tail = (prob.scale, *args) if kind == "window" else (*args, prob.scale)
    fn(q, *cache, bt, None if uniform else cu, lens, *tail, out, ws, num_workers=workers, err_word=err,
       new_per_seq=uniform)
    assert err.item() == err_is
    return out


LENS = [1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 257, 500, 700, 1100]


# ------------------------------------------------------------------------------------------ one new token
@pytest.mark.parametrize("cache", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 16), (64, 0), (100, 5), (128, 130), (600, 40),
                                          (1 << 30, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 4096)])
def test_decode_windows(cache, window, sinks):
    sees = [window_sees(L, 1, window, sinks) for L in LENS]
    prob = Problem(cache, sees, 16, 8, 128, 16 if window != 100 else 64, seed=window % 97 + sinks)
    for workers in (0, 40):
        check(decode(prob, window, sinks, workers), prob, f"workers {workers}")


@pytest.mark.parametrize("cache,Hq,Hkv,D,bs", [
    ("bf16", 4, 2, 64, 8), ("bf16", 14, 2, 64, 16), ("bf16", 16, 16, 64, 32), ("bf16", 16, 1, 128, 16),
    ("bf16", 15, 5, 128, 128), ("bf16", 22, 11, 64, 256), ("bf16", 9, 1, 64, 512), ("bf16", 3, 3, 128, 1024),
    ("fp8", 4, 2, 64, 8), ("fp8", 8, 1, 128, 32), ("fp8", 6, 3, 64, 256), ("fp8", 22, 11, 128, 16),
    ("int8", 4, 2, 64, 16), ("int8", 16, 1, 128, 32), ("int8", 14, 2, 128, 64), ("int8", 12, 4, 64, 1024),
    ("int8", 13, 13, 64, 16), ("int8", 15, 5, 128, 256)])
def test_decode_layouts(cache, Hq, Hkv, D, bs):
    for window, sinks in ((37, 5), (300, 0)):
        prob = Problem(cache, [window_sees(L, 1, window, sinks) for L in LENS], Hq, Hkv, D, bs, seed=Hq + D + bs)
        check(decode(prob, window, sinks), prob, f"{window} {sinks}")


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int8"])
def test_decode_of_empty_and_long_sequences(cache):
    """Length 0 gives zeros; a long sequence is split over many CTAs, whose pieces meet inside the window."""
    window, sinks = 20000, 700
    sees = [window_sees(L, min(L, 1), window, sinks) for L in (30000, 3, 21000, 800)]
    prob = Problem(cache, sees, 8, 2, 128, 64, seed=3)
    check(decode(prob, window, sinks), prob, "long")
    q, c, bt, lens, _ = prob.cuda()
    lens[1] = 0
    out = decode(prob, window, sinks, dev=(q, c, bt, lens, None))
    assert not out[1].any()


def test_many_sequences_and_one_workspace():
    """More sequences than split slots, counters outside the fixed region, and one workspace for calls of other kinds and
    sizes in turn."""
    rng = np.random.default_rng(1)
    ws = pkv.alloc_workspace(2100, 16, 8, 64)
    for B, window, sinks in ((2100, 40, 2), (3, 9, 0), (700, 130, 17)):
        lens = rng.integers(1, 300, B)
        prob = Problem("bf16", [window_sees(int(L), 1, window, sinks) for L in lens], 16, 8, 64, 16, seed=B)
        check(decode(prob, window, sinks, ws=ws), prob, f"B {B}")
        full = Problem("bf16", [window_sees(int(L), 1, 1 << 20, 0) for L in lens], 16, 8, 64, 16, seed=B)
        q, c, bt, ld, _ = full.cuda()
        out = torch.empty_like(q)
        pkv.paged_decode(q, *c, bt, ld, full.scale, out, ws)
        check(out, full, "plain decode between")


def test_a_window_over_all_is_the_plain_decode():
    prob = Problem("bf16", [window_sees(L, 1, 5000, 0) for L in LENS], 16, 8, 128, 16, seed=5)
    q, c, bt, lens, _ = dev = prob.cuda()
    for workers in (1, 33):
        ws = pkv.alloc_workspace(len(LENS), 16, 8, 128)
        out = torch.empty_like(q)
        pkv.paged_decode(q, *c, bt, lens, prob.scale, out, ws, num_workers=workers)
        assert torch.equal(out, decode(prob, 5000, 0, workers, dev=dev))


# ------------------------------------------------------------------------------------------ several new tokens
@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("n", [1, 2, 5, 8, 13, 16, 17, 64, 130])
@pytest.mark.parametrize("window,sinks,bs", [(1, 0, 16), (13, 3, 128), (100, 1, 256), (400, 140, 32)])
def test_attention_windows(cache, n, window, sinks, bs):
    lens = [max(L, n) for L in LENS]
    prob = Problem(cache, [window_sees(L, n, window, sinks) for L in lens], 16, 8, 128, bs, seed=n + window)
    for workers, uniform in ((0, n), (24, 0)):
        out = attend(prob, (window, sinks), uniform=uniform, workers=workers)
        check(out, prob, f"workers {workers}", long_runs=n > 8 or not uniform)


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(4, 2, 64, 16), (14, 2, 64, 128), (16, 1, 128, 256), (15, 5, 64, 16),
                                         (8, 8, 64, 256), (12, 4, 128, 512), (32, 8, 64, 128)])
def test_attention_ragged(cache, Hq, Hkv, D, bs):
    """Single tokens, chunks and whole prompts in one call."""
    lens, new = [700, 1, 33, 300, 1000, 257, 50, 900], [700, 1, 5, 300, 1, 64, 50, 129]
    for window, sinks in ((50, 4), (256, 0)):
        prob = Problem(cache, [window_sees(L, n, window, sinks) for L, n in zip(lens, new)], Hq, Hkv, D, bs, seed=Hq + bs)
        check(attend(prob, (window, sinks)), prob, f"{window} {sinks}", long_runs=True)


def test_attention_with_sequences_without_new_tokens():
    lens, new = [40, 0, 300, 20, 0], [3, 0, 0, 20, 0]
    prob = Problem("bf16", [window_sees(L, n, 16, 2) for L, n in zip(lens, new)], 8, 4, 64, 16, seed=2)
    check(attend(prob, (16, 2)), prob, "some without", long_runs=True)


# ------------------------------------------------------------------------------------------ trees
@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("n,words", [(1, 1), (2, 1), (7, 3), (8, 1), (13, 1), (16, 2), (25, 1), (32, 1), (33, 2),
                                     (64, 2), (100, 4), (150, 5)])
def test_trees(cache, n, words):
    rng = np.random.default_rng(n)
    lens = [max(L, n) for L in LENS]
    masks = random_trees([n] * len(lens), words, rng)
    sees = [tree_sees(L, n, masks[b * n:(b + 1) * n]) for b, L in enumerate(lens)]
    for Hq, Hkv, D, bs in ((16, 8, 128, 16), (8, 1, 64, 256)):
        prob = Problem(cache, sees, Hq, Hkv, D, bs, seed=n + Hq)
        md = torch.from_numpy(masks).cuda()
        for workers, uniform in ((0, n), (24, 0)):
            out = attend(prob, (md,), "tree", uniform=uniform, workers=workers)
            check(out, prob, f"heads {Hq} workers {workers}", long_runs=n * Hq > 16 * Hkv or not uniform)


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(14, 2, 64, 16), (16, 8, 128, 128), (15, 5, 128, 32), (16, 16, 64, 256),
                                         (4, 2, 64, 512)])
def test_ragged_trees(cache, Hq, Hkv, D, bs):
    rng = np.random.default_rng(Hq)
    lens, new = [200, 64, 500, 1, 90, 300, 129, 31], [64, 64, 1, 1, 0, 17, 90, 31]
    masks = random_trees(new, 3, rng)
    cu = np.concatenate([[0], np.cumsum(new)])
    sees = [tree_sees(L, n, masks[a:a + n]) for L, n, a in zip(lens, new, cu)]
    prob = Problem(cache, sees, Hq, Hkv, D, bs, seed=bs)
    check(attend(prob, (torch.from_numpy(masks).cuda(),), "tree"), prob, "ragged", long_runs=True)


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("n", [3, 12, 40])
def test_rows_that_see_nothing_give_zeros(cache, n):
    """A draft at the start of a sequence: empty masks, and nodes that see others but not themselves."""
    rng = np.random.default_rng(n)
    lens = [n, n, n + 1, n + 20, n]
    masks = random_trees([n] * 5, 2, rng, noise=False)
    masks[:n] = 0                                 # all of sequence 0
    masks[n:2 * n:2] = 0                          # every second row of sequence 1
    masks[4 * n + 2, :] = 1                       # node 2 sees the root alone
    sees = [tree_sees(L, n, masks[b * n:(b + 1) * n]) for b, L in enumerate(lens)]
    # (keys that no row sees still belong to the draft: they are real rows)
    for b in (0, 1):
        sees[b] = np.zeros_like(sees[b]) if b == 0 else sees[b]
    prob = Problem(cache, [tree_sees(L, n, random_trees([n], 2, rng, noise=False)) for L in lens], 16, 8, 64, 16, seed=n)
    prob.sees = sees
    for uniform in (n, 0):
        out = attend(prob, (torch.from_numpy(masks).cuda(),), "tree", uniform=uniform)
        assert not out[:n].any() and not out[n:2 * n:2].any()
        check(out, prob, "some empty", long_runs=n > 8 or not uniform)


@pytest.mark.parametrize("n", [1, 5, 8, 16, 40])
def test_a_chain_is_the_plain_attention(n):
    lens = [max(L, n) for L in LENS]
    chain = np.tril(np.ones((n, 64), np.uint8))
    mask = np.packbits(chain, axis=1, bitorder="little").view(np.int32)
    masks = torch.from_numpy(np.tile(mask, (len(lens), 1))).cuda()
    prob = Problem("bf16", [window_sees(L, n, 1 << 20, 0) for L in lens], 16, 8, 128, 128, seed=n)
    dev = prob.cuda()
    for uniform in (n, 0):
        tree, window = (attend(prob, *a, workers=20, dev=dev, uniform=uniform) for a in (((masks,), "tree"), ((1 << 20, 0),)))
        assert torch.equal(tree, window)
        check(tree, prob, "chain", long_runs=n > 8 or not uniform)
        if 1 < n <= 8 and uniform:  # (the others run on another kernel than the plain call, whose sums have another order)
            q, c, bt, ld, cu = dev
            ws = pkv.alloc_attention_workspace(q.shape[0], 16, 8, 128)
            out = torch.empty_like(q)
            pkv.paged_attention(q, *c, bt, cu, ld, prob.scale, out, ws, num_workers=20, new_per_seq=n)
            assert torch.equal(out, tree)


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(16, 8, 128, 256), (4, 1, 64, 16), (15, 5, 128, 32)])
@pytest.mark.parametrize("lens,new", [([30000], [25]), ([9000, 700, 20000], [33, 1, 150]), ([12345, 4000], [64, 64])])
def test_few_long_sequences(Hq, Hkv, D, bs, lens, new):
    """Segments of many pieces, merged by a kernel of their own."""
    masks = random_trees(new, 5, np.random.default_rng(3))
    cu = np.concatenate([[0], np.cumsum(new)])
    prob = Problem("bf16", [tree_sees(L, n, masks[a:a + n]) for L, n, a in zip(lens, new, cu)], Hq, Hkv, D, bs, seed=Hq)
    md, dev = torch.from_numpy(masks).cuda(), prob.cuda()
    ws = pkv.alloc_attention_workspace(sum(new), Hq, Hkv, D)
    for workers in (0, 100):
        out = attend(prob, (md,), "tree", workers=workers, dev=dev, ws=ws)
        check(out, prob, f"workers {workers}", long_runs=True)
        assert torch.equal(out, attend(prob, (md,), "tree", workers=workers, dev=dev, ws=ws))


@pytest.mark.parametrize("Hq,Hkv,D,B,top", [(16, 8, 128, 40, 4000), (14, 2, 64, 48, 3000), (32, 8, 128, 16, 4000)])
def test_many_long_sequences(Hq, Hkv, D, B, top):
    """Segments of several pieces, more of them than CTAs: the CTAs that complete them merge.  Pages end in the middle of
    a unit, and what lies behind a sequence's last token is not a number: every copy has to have landed before those
    rows are overwritten, time after time."""
    rng = np.random.default_rng(B)
    lens = [int(L) for L in rng.integers(500, top, B)]
    new = [20] * B
    masks = random_trees(new, 1, rng)
    prob = Problem("bf16", [tree_sees(L, 20, masks[20 * b:20 * b + 20]) for b, L in enumerate(lens)], Hq, Hkv, D, 256, seed=B)
    md, dev = torch.from_numpy(masks).cuda(), prob.cuda()
    ws = pkv.alloc_attention_workspace(20 * B, Hq, Hkv, D)
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for uniform in (20, 0):
        first = attend(prob, (md,), "tree", uniform=uniform, dev=dev, ws=ws)
        check(first, prob, "many", long_runs=True)
        for i in range(20):
            if i % 2:
                big.fill_(i)  # (the caches have to come from memory again)
            assert torch.equal(first, attend(prob, (md,), "tree", uniform=uniform, dev=dev, ws=ws))
    prob.sees = [window_sees(L, 20, 2000, 70) for L in lens]
    check(attend(prob, (2000, 70), dev=dev, ws=ws), prob, "windows", long_runs=True)


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("B,Hkv", [(400, 8), (300, 2), (70, 1), (2200, 8)])
def test_most_sequences_without_new_tokens(cache, B, Hkv):
    """A workspace for the rows does, whatever the number of sequences: what lies behind it stays."""
    lens = [5000 + 13 * b if b % (B // 10) == 3 else 40 for b in range(B)]
    new = [1 + b % 3 if L > 40 else 0 for b, L in enumerate(lens)]
    masks = random_trees(new, 1, np.random.default_rng(B))
    cu = np.concatenate([[0], np.cumsum(new)])
    prob = Problem(cache, [tree_sees(L, n, masks[a:a + n]) for L, n, a in zip(lens, new, cu)], 2 * Hkv, Hkv, 64, 64, seed=B)
    n = pkv.alloc_attention_workspace(sum(new), 2 * Hkv, Hkv, 64).numel()
    whole = torch.zeros(n + (1 << 22), dtype=torch.uint8, device="cuda")
    whole[n:] = 0xA5
    dev, md = prob.cuda(), torch.from_numpy(masks).cuda()
    first = attend(prob, (md,), "tree", dev=dev, ws=whole[:n])
    check(first, prob, "few rows", long_runs=True)
    for workers in (0, 4096):
        check(attend(prob, (md,), "tree", dev=dev, ws=whole[:n], workers=workers), prob, f"workers {workers}", long_runs=True)
    assert (whole[n:] == 0xA5).all()


def test_more_segments_than_the_fixed_counters():
    """2100 sequences of one node each and more on 8 kv heads: counters by row, cleared by the call."""
    B = 2100
    lens, new = [1400 + b % 5 if b % 50 == 0 else 30 for b in range(B)], [1 + b % 3 for b in range(B)]
    masks = random_trees(new, 1, np.random.default_rng(1))
    cu = np.concatenate([[0], np.cumsum(new)])
    prob = Problem("bf16", [tree_sees(L, n, masks[a:a + n]) for L, n, a in zip(lens, new, cu)], 8, 8, 64, 32, seed=1)
    dev, md = prob.cuda(), torch.from_numpy(masks).cuda()
    ws = pkv.alloc_attention_workspace(sum(new), 8, 8, 64)
    ws.random_(generator=torch.Generator(device="cuda").manual_seed(0))
    ws[:1 << 18] = 0  # (the part that has to be zero before the first use)
    first = attend(prob, (md,), "tree", dev=dev, ws=ws)
    check(first, prob, "many", long_runs=True)
    assert torch.equal(first, attend(prob, (md,), "tree", dev=dev, ws=ws))


# ------------------------------------------------------------------------------------------ arguments of every kind
@pytest.mark.parametrize("cache", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("scale", [-0.07, 0.0])
def test_scales_of_either_sign(cache, scale):
    lens = [3, 64, 130, 700]
    prob = Problem(cache, [window_sees(L, 1, 90, 4) for L in lens], 16, 8, 64, 32, seed=1)
    prob.scale = scale
    check(decode(prob, 90, 4), prob, "decode")
    for n in (3, 40) if cache != "fp8" else ():
        prob = Problem(cache, [window_sees(L, min(L, n), 90, 4) for L in lens], 16, 8, 64, 32, seed=n)
        prob.scale = scale
        check(attend(prob, (90, 4)), prob, f"window {n}", long_runs=True)
        masks = random_trees([min(L, n) for L in lens], 2, np.random.default_rng(n))
        cu = np.concatenate([[0], np.cumsum(prob.new)])
        prob.sees = [tree_sees(L, m, masks[a:a + m]) for L, m, a in zip(lens, prob.new, cu)]
        prob = Problem(cache, prob.sees, 16, 8, 64, 32, seed=n)
        prob.scale = scale
        check(attend(prob, (torch.from_numpy(masks).cuda(),), "tree"), prob, f"tree {n}", long_runs=True)


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("n", [4, 33])
def test_outputs_queries_and_masks_at_their_least_alignment(cache, n):
    """q and out begin 16 bytes after a boundary of 32, the mask 4 after one of 8; what surrounds out stays."""
    lens = [40, 300, 77]
    masks = random_trees([n] * 3, 2, np.random.default_rng(n))
    prob = Problem(cache, [tree_sees(L, n, masks[b * n:b * n + n]) for b, L in enumerate(lens)], 14, 2, 64, 16, seed=n)
    q, c, bt, ld, cu = prob.cuda()
    T = q.shape[0]
    place = lambda t, pad: torch.full((t.numel() + 2 * pad,), -7, dtype=t.dtype, device="cuda")
    qb, ob, mb = place(q, 8), place(q, 8), place(torch.from_numpy(masks), 1)
    qb[8:-8], mb[1:-1] = q.flatten(), torch.from_numpy(masks).cuda().flatten()
    view = lambda b: b[8:-8].view(T, 14, 64)
    ws = pkv.alloc_attention_workspace(T, 14, 2, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    fn = pkv.paged_attention_tree if cache == "bf16" else pkv.paged_attention_tree_i8
    for uniform in (0, n):
        ob.fill_(-7)
        fn(view(qb), *c, bt, None if uniform else cu, ld, mb[1:-1].view(T, 2), prob.scale, view(ob), ws, err_word=err,
           new_per_seq=uniform)
        assert err.item() == 0 and (ob[:8] == -7).all() and (ob[-8:] == -7).all()
        check(view(ob), prob, f"uniform {uniform}", long_runs=True)


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("cu", [[0, 40, 20, 90], [0, 90, 90, 10, 90], [3, 30, 90], [0, -3, 90], [0, 30, 60], [0, 0, 0],
                                [0, 30, 95], [0, 10, 90]])
def test_offsets_that_do_not_fit(cache, cu):
    """Flagged; rows of no sequence, of sequences that do not fit, or of offsets out of order give zeros, and the
    others what they give alone."""
    T, Hq, Hkv, D = 90, 8, 2, 64
    lens = [70] * (len(cu) - 1)
    prob = Problem(cache, [window_sees(70, 1, 4000, 0)] * len(lens), Hq, Hkv, D, 16, seed=5)
    _, c, bt, ld, _ = prob.cuda()
    prob.q = torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    order = cu[0] == 0 and all(a <= b for a, b in zip(cu, cu[1:]))
    prob.sees, want_zero = [], []
    for a, b, L in zip(cu, cu[1:], lens):
        if order:
            good = b - a <= L and b <= T
            prob.sees.append(window_sees(L, b - a, 33, 2) if good else np.zeros((min(b, T) - a, L), bool))
            want_zero += range(a, min(b, T)) if not good else ()
    if not order:
        prob.sees, prob.bt, want_zero = [np.zeros((T, 70), bool)], prob.bt[:1], range(T)
    elif cu[-1] < T:
        prob.sees.append(np.zeros((T - cu[-1], 70), bool))
        prob.bt = np.concatenate([prob.bt, prob.bt[:1]])
        want_zero += range(cu[-1], T)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = attend(prob, (33, 2), err_is=pkv.ERR_CONTEXT_RANGE, dev=(prob.q.cuda(), c, bt, ld, off))
    assert not out[list(want_zero)].any()
    check(out, prob, str(cu), long_runs=True)


# ------------------------------------------------------------------------------------------ what the device refuses
def test_bad_pages_lengths_and_offsets_are_flagged():
    prob = Problem("bf16", [window_sees(L, 1, 30, 2) for L in (100, 200)], 4, 2, 64, 16, seed=0)
    q, c, bt, lens, _ = prob.cuda()
    ws = pkv.alloc_workspace(2, 4, 2, 64)
    for bad, flag in (((0, 0), pkv.ERR_BLOCK_RANGE), ((1, 11), pkv.ERR_BLOCK_RANGE), ((0, 3), 0)):
        t, err = bt.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        t[bad] = 1 << 20
        pkv.paged_decode_window(q, *c, t, lens, 0.1, 30, 2, torch.empty_like(q), ws, err_word=err)
        assert err.item() == flag
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"))
    pkv.paged_decode_window(q, *c, bt, torch.tensor([-1, 1 << 20], dtype=torch.int32, device="cuda"), 0.1, 30, 2, out, ws,
                            err_word=err)
    assert err.item() == pkv.ERR_CONTEXT_RANGE and not out.any()


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("n,m", [(40, 20), (70, 33)])
def test_more_nodes_than_the_mask_holds(cache, n, m):
    masks = random_trees([n, m], -(-m // 32), np.random.default_rng(0), noise=False) if n <= 32 else \
        np.concatenate([np.full((n, -(-m // 32)), -1, np.int32), random_trees([m], -(-m // 32), np.random.default_rng(0))])
    sees = [window_sees(100, n, 200, 0), tree_sees(90, m, masks[n:])]
    prob = Problem(cache, sees, 8, 4, 64, 16, seed=n)
    out = attend(prob, (torch.from_numpy(masks).cuda(),), "tree", err_is=pkv.ERR_CONTEXT_RANGE if n > 32 * masks.shape[1]
                 else 0)
    if n > 32 * masks.shape[1]:
        assert not out[:n].any()
        prob.sees[0] = np.zeros_like(sees[0])
    check(out, prob, "the other sequence", long_runs=True)


# ------------------------------------------------------------------------------------------ streams and graphs
def test_captured_calls_replay_with_other_contents():
    """One graph of a windowed decode, a windowed chunk and a tree over one workspace, replayed as the sequences grow and
    their pages leave the window."""
    Hq, Hkv, D, bs, B, n = 16, 8, 128, 16, 6, 20
    ws = pkv.alloc_attention_workspace(B * n, Hq, Hkv, D)
    probs = []
    for step in range(3):
        rng = np.random.default_rng(step)
        lens = [30 + 47 * b + 90 * step for b in range(B)]
        masks = random_trees([n] * B, 1, rng)
        probs.append((
            Problem("bf16", [window_sees(L, 1, 60, 4) for L in lens], Hq, Hkv, D, bs, seed=step),
            Problem("bf16", [window_sees(L, n, 60, 4) for L in lens], Hq, Hkv, D, bs, seed=step + 10),
            Problem("bf16", [tree_sees(L, n, masks[b * n:(b + 1) * n]) for b, L in enumerate(lens)], Hq, Hkv, D, bs,
                    seed=step + 20), masks))
    NB, mb = 400, 64
    state = []
    for i in range(3):
        T = B if i == 0 else B * n
        state.append(dict(q=torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
                          c=[torch.zeros(NB, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)],
                          bt=torch.full((B, mb), -1, dtype=torch.int32, device="cuda"),
                          lens=torch.zeros(B, dtype=torch.int32, device="cuda"),
                          out=torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")))
    md = torch.zeros(B * n, 1, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def load(group):
        for st, pr in zip(state, group[:3]):
            q, c, bt, lens, _ = pr.cuda()
            st["q"].copy_(q)
            for dst, src in zip(st["c"], c):
                dst[:src.shape[0]] = src
            st["bt"].fill_(-1)
            st["bt"][:, :bt.shape[1]] = bt
            st["lens"].copy_(lens)
        md.copy_(torch.from_numpy(group[3]))

    def call():
        a, b, c = state
        s = D ** -0.5
        pkv.paged_decode_window(a["q"], *a["c"], a["bt"], a["lens"], s, 60, 4, a["out"], ws, err_word=err)
        pkv.paged_attention_window(b["q"], *b["c"], b["bt"], None, b["lens"], s, 60, 4, b["out"], ws, new_per_seq=n,
                                   err_word=err)
        pkv.paged_attention_tree(c["q"], *c["c"], c["bt"], None, c["lens"], md, s, c["out"], ws, new_per_seq=n,
                                 err_word=err)

    load(probs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for group in (probs[1], probs[2], probs[0]):
        load(group)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert err.item() == 0
        for st, pr in zip(state, group[:3]):
            check(st["out"], pr, "replayed", long_runs=True)


def test_two_streams_with_their_own_workspaces():
    probs = [Problem("bf16", [window_sees(900 + 10 * i, 1, 300, 8) for i in range(40)], 16, 8, 128, 16, seed=s)
             for s in range(2)]
    dev = [p.cuda() for p in probs]
    ws = [pkv.alloc_workspace(40, 16, 8, 128) for _ in probs]
    outs = [torch.empty_like(d[0]) for d in dev]
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, d, w, o, s in zip(probs, dev, ws, outs, streams):
            pkv.paged_decode_window(d[0], *d[1], d[2], d[3], p.scale, 300, 8, o, w, stream=s)
    torch.cuda.synchronize()
    for p, o in zip(probs, outs):
        check(o, p, "beside another")


def test_fixed_splits_repeat_bit_for_bit():
    prob = Problem("bf16", [window_sees(L, 30, 333, 20) for L in (2000, 700, 90, 1200)], 16, 8, 128, 128, seed=1)
    dev = prob.cuda()
    first = attend(prob, (333, 20), workers=50, dev=dev)
    for _ in range(3):
        assert torch.equal(first, attend(prob, (333, 20), workers=50, dev=dev))


def test_bindings_refuse():
    prob = Problem("bf16", [window_sees(20, 1, 5, 0)] * 3, 4, 2, 64, 16, seed=0)
    q, c, bt, lens, cu = prob.cuda()
    ws, aws = pkv.alloc_workspace(3, 4, 2, 64), pkv.alloc_attention_workspace(3, 4, 2, 64)
    out = torch.zeros_like(q)
    i8 = pkv.alloc_i8_cache(4, 16, 2, 64)
    mask = torch.ones(3, 1, dtype=torch.int32, device="cuda")
    dec = lambda *a, **k: pkv.paged_decode_window(*a, **k)
    with pytest.raises(ValueError, match="int|Byte|BFloat"):
        dec(q, i8[0], i8[1], bt, lens, 0.1, 5, 0, out, ws)
    with pytest.raises(ValueError, match="shape"):
        dec(q[:2], *c, bt, lens, 0.1, 5, 0, out[:2], ws)
    with pytest.raises(ValueError, match="scales"):
        pkv.paged_decode_window_i8(q, i8[0], i8[1], None, bt, lens, 0.1, 5, 0, out, ws)
    with pytest.raises(ValueError, match="window"):
        dec(q, *c, bt, lens, 0.1, 1 << 31, 0, out, ws)
    with pytest.raises(TypeError):
        dec(q, *c, bt, lens, 0.1, 2.5, 0, out, ws)
    for w, s in ((0, 0), (-1, 3), (4, -1)):
        with pytest.raises(pkv.PkvError) as e:
            dec(q, *c, bt, lens, 0.1, w, s, out, ws)
        assert e.value.status == pkv.EINVAL
    with pytest.raises(ValueError, match="tree_mask"):
        pkv.paged_attention_tree(q, *c, bt, cu, lens, None, 0.1, out, aws)
    with pytest.raises(ValueError, match="tree"):
        pkv.paged_attention_tree(q, *c, bt, cu, lens, mask[:2], 0.1, out, aws)
    with pytest.raises(ValueError, match="tree_mask"):
        pkv.paged_attention_tree(q, *c, bt, cu, lens, mask.long(), 0.1, out, aws)
    with pytest.raises(ValueError, match="tree"):
        pkv.paged_attention_tree(q, *c, bt, None, lens, mask, 0.1, out, aws)
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_window(q, *c, bt, cu, lens, 0.1, 5, 0, out, aws[:1024])
    assert not out.any()
