"""GPU tests of windowed and tree calls at their edges: drafted nodes that nobody sees, lengths and table entries that do
not fit, scale blocks of zeros and of no numbers, keys that are not finite, long tables, and the weights' precision when
few new tokens come by offsets.  Bounds as in test_gpu_masks.py.
"""
import numpy as np
import pytest
import torch

from mask_reference import SB, Problem, random_trees, tree_sees, window_sees
from paged_kv_cache_62_gb300 import pkv
from test_gpu_masks import attend, check, decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def only(prob, keep):
    """The problem of some sequences of another one, over the same cache, and the rows of theirs."""
    part = object.__new__(Problem)
    part.__dict__.update(prob.__dict__)
    cu = np.concatenate([[0], np.cumsum(prob.new)])
    rows = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in keep]) if keep else np.zeros(0, int)
    part.sees, part.bt = [prob.sees[b] for b in keep], prob.bt[keep]
    part.lens, part.new, part.q = [prob.lens[b] for b in keep], [prob.new[b] for b in keep], prob.q[rows]
    return part, rows


# ------------------------------------------------------------------------------------------ nodes that nobody sees
def padded_trees(new, pads, words, rng):
    """Trees whose last pads[b] nodes are no node's to see, not even their own; they see what their parents see."""
    masks, r = random_trees(new, words, rng), 0
    for n, k in zip(new, pads):
        bits = np.unpackbits(masks[r:r + n].view(np.uint8), axis=1, bitorder="little")
        bits[:, n - k:n] = 0
        masks[r:r + n] = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
        r += n
    return masks


@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(16, 8, 128, 256), (8, 1, 64, 16), (15, 5, 64, 32)])
@pytest.mark.parametrize("n,pad", [(2, 1), (5, 3), (8, 6), (20, 17), (40, 24), (70, 40), (100, 99)])
def test_nodes_that_nobody_sees_may_hold_anything(cache, Hq, Hkv, D, bs, n, pad):
    """Places of a batch of trees that a sequence's tree leaves unused: their K, V and scales are not numbers."""
    lens = [n, n + 1, n + 11, max(n, 16) + 5, 64 + n, 133 + n, 700, 1100]
    pads = [pad if b % 3 else max(pad - 1, 0) for b in range(len(lens))]
    masks = padded_trees([n] * len(lens), pads, 4, np.random.default_rng(n))
    sees = [tree_sees(L, n, masks[b * n:b * n + n]) for b, L in enumerate(lens)]
    prob = Problem(cache, sees, Hq, Hkv, D, bs, seed=n + Hq, bad=0)
    md, dev = torch.from_numpy(masks).cuda(), prob.cuda()
    for workers, uniform in ((0, n), (0, 0), (40, n), (40, 0)):
        out = attend(prob, (md,), "tree", uniform=uniform, workers=workers, dev=dev)
        check(out, prob, f"uniform {uniform} workers {workers}", long_runs=True)


# ------------------------------------------------------------------------------------------ lengths
@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("n", [1, 3, 30])
@pytest.mark.parametrize("bad", [0, -1, 1 << 20, -(1 << 31)])
def test_lengths_that_do_not_fit(kind, cache, n, bad):
    """Fewer keys than new tokens, negative lengths and lengths beyond the table: flagged, zeros, the others unharmed;
    the same with a fixed number of new tokens and with offsets."""
    lens, wrong = [40, 300, 77, 64], [1, 3]
    if kind == "window":
        prob = Problem(cache, [window_sees(L, n, 50, 3) for L in lens], 16, 8, 64, 16, seed=n)
        args = (50, 3)
    else:
        masks = random_trees([n] * 4, 1, np.random.default_rng(n))
        prob = Problem(cache, [tree_sees(L, n, masks[b * n:b * n + n]) for b, L in enumerate(lens)], 16, 8, 64, 16, seed=n)
        args = (torch.from_numpy(masks).cuda(),)
    q, c, bt, ld, cu = prob.cuda()
    ld[wrong] = bad
    good, rows = only(prob, [0, 2])
    for uniform in (n, 0):
        out = attend(prob, args, kind, uniform=uniform, err_is=pkv.ERR_CONTEXT_RANGE, dev=(q, c, bt, ld, cu))
        for b in wrong:
            assert not out[b * n:b * n + n].any(), uniform
        check(out[rows], good, f"uniform {uniform}", long_runs=True)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("bad", [-1, 1 << 20, -(1 << 31)])
def test_decode_lengths_that_do_not_fit(cache, bad):
    prob = Problem(cache, [window_sees(L, 1, 50, 3) for L in (40, 300, 77, 64)], 16, 8, 64, 16, seed=1)
    q, c, bt, ld, _ = prob.cuda()
    ld[1] = bad
    out, err = torch.full_like(q, float("nan")), torch.zeros(1, dtype=torch.int32, device="cuda")
    name = {"bf16": "", "fp8": "_fp8", "int8": "_i8"}[cache]
    getattr(pkv, "paged_decode_window" + name)(q, *c, bt, ld, prob.scale, 50, 3, out, pkv.alloc_workspace(4, 16, 8, 64),
                                               err_word=err)
    assert err.item() == pkv.ERR_CONTEXT_RANGE and not out[1].any()
    good, rows = only(prob, [0, 2, 3])
    check(out[rows], good, "others")


# ------------------------------------------------------------------------------------------ table entries
@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("n", [1, 4, 33, 90])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(16, 8, 64, 16), (6, 2, 128, 128)])
def test_table_entries_out_of_range(cache, kind, n, Hq, Hkv, D, bs):
    """An entry that names no block is flagged where a query needs it, at any place of the sequence, and not looked at
    elsewhere; the other sequences get what they get without it."""
    lens, masks = [400, 300, 500, 277], None
    if kind == "window":
        sees, args = [window_sees(L, n, 60, 3) for L in lens], (60, 3)
    else:
        masks = random_trees([n] * 4, 3, np.random.default_rng(n))
        sees = [tree_sees(L, n, masks[b * n:b * n + n]) for b, L in enumerate(lens)]
        args = (torch.from_numpy(masks).cuda(),)
    prob = Problem(cache, sees, Hq, Hkv, D, bs, seed=n + bs)
    q, c, bt, ld, cu = prob.cuda()
    NB = c[0].shape[0]
    good, rows = only(prob, [0, 1, 3])
    needed = [p for p in range(-(-lens[2] // bs)) if prob.bt[2, p] >= 0]
    spare = [p for p in range(prob.bt.shape[1]) if prob.bt[2, p] < 0]
    for uniform in (n, 0):
        for page, entry in zip((needed[0], needed[-1], needed[len(needed) // 2]), (NB, -1, 2 ** 31 - 1)):
            t = bt.clone()
            t[2, page] = entry
            out = attend(prob, args, kind, uniform=uniform, err_is=pkv.ERR_BLOCK_RANGE, dev=(q, c, t, ld, cu))
            check(out[rows], good, f"uniform {uniform} page {page}", long_runs=True)
        t = bt.clone()
        t[2, spare] = 2 ** 31 - 1
        check(attend(prob, args, kind, uniform=uniform, dev=(q, c, t, ld, cu)), prob, "spare", long_runs=True)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int8"])
def test_decode_table_entries_out_of_range(cache):
    prob = Problem(cache, [window_sees(L, 1, 60, 3) for L in (400, 300, 500, 277)], 16, 8, 64, 16, seed=1)
    q, c, bt, ld, _ = prob.cuda()
    NB, good = c[0].shape[0], only(prob, [0, 1, 3])
    name = {"bf16": "", "fp8": "_fp8", "int8": "_i8"}[cache]
    ws = pkv.alloc_workspace(4, 16, 8, 64)
    for page, entry, flag in ((0, NB, 1), (31, -1, 1), (29, 2 ** 31 - 1, 1), (10, 2 ** 31 - 1, 0)):
        t = bt.clone()
        t[2, page] = entry
        out, err = torch.full_like(q, float("nan")), torch.zeros(1, dtype=torch.int32, device="cuda")
        getattr(pkv, "paged_decode_window" + name)(q, *c, t, ld, prob.scale, 60, 3, out, ws, err_word=err)
        assert err.item() == (pkv.ERR_BLOCK_RANGE if flag else 0)
        check(out[good[1]], good[0], f"page {page}")
        if not flag:
            check(out, prob, "spare")


# ------------------------------------------------------------------------------------------ scale blocks
def scale_problem(kind, n, Hq, Hkv, D, bs, change, seed):
    """An int8 problem whose scales `change` alters; the 64-bit values follow."""
    lens = [max(n, 90), 300 + n, 517]
    if kind == "window":
        sees, args = [window_sees(L, n, 130, 20) for L in lens], (130, 20)
    else:
        masks = random_trees([n] * 3, 3, np.random.default_rng(n), noise=False)
        sees = [tree_sees(L, n, masks[b * n:b * n + n]) for b, L in enumerate(lens)]
        args = (torch.from_numpy(masks).cuda(),)
    prob = Problem("int8", sees, Hq, Hkv, D, bs, seed)
    change(prob)
    wide = prob.sc.double()
    wide = torch.where(wide.abs() < 2.0 ** -104, 0.0, wide).repeat_interleave(SB, 1)  # smaller V scales count as zero
    prob.kd, prob.vd = prob.kc.double() * wide[..., 0:1], prob.vc.double() * wide[..., 1:2]
    return prob, args


@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("n", [1, 6, 40, 90])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(16, 8, 128, 16), (8, 1, 64, 64)])
@pytest.mark.parametrize("which", [(0,), (1,), (0, 1)])
def test_scale_blocks_of_zeros_under_a_mask(kind, n, Hq, Hkv, D, bs, which):
    """K blocks of zeros score zero, V blocks of zeros (or of scales that count as zero) add weight and no values.

    A code enters the 16-row tiles' output product 1152 too large and a second product takes that off again: two
    roundings at 1152 times the weights, 2^-23 of it each where an accumulator truncates, leave less than 2^-11 of a
    code.  Beside codes of ordinary blocks the bound's other terms cover that; a row that sees blocks of zeros alone
    has nothing else, so the largest V scale's 2^-11 is added."""
    rng = np.random.default_rng(n)

    def change(prob):
        for i in which:
            hit = torch.from_numpy(rng.random(prob.sc.shape[:3]) < 0.4)
            small = torch.from_numpy(rng.random(hit.shape) < 0.3) & bool(i)
            old = prob.sc[..., i]
            prob.sc[..., i] = torch.where(hit & ~old.isnan(), torch.where(small, 2.0 ** -110, 0.0), old)

    prob, args = scale_problem(kind, n, Hq, Hkv, D, bs, change, n + Hq)
    want, mag = prob.want()
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag + 2.0 ** -11 * prob.sc[..., 1].nan_to_num().max().item()
    dev = prob.cuda()
    outs = [attend(prob, args, kind, uniform=uniform, dev=dev) for uniform in (n, 0)]
    if n == 1 and kind == "window":
        outs.append(decode(prob, *args, dev=dev))
    for out in outs:
        off = (out.cpu().double() - want).abs() - bound
        assert off.max() <= 0, off.max().item()


@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("n", [1, 6, 40, 90])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("i", [0, 1])
def test_a_scale_block_that_is_no_number_spoils_its_readers_alone(kind, n, what, i):
    """The block of a sequence's first keys (a sink's) and one kv head: the queries of that head give no numbers, the
    other heads and sequences what they give without it."""
    clean, args = scale_problem(kind, n, 16, 4, 64, 16, lambda prob: None, n)
    dirty, _ = scale_problem(kind, n, 16, 4, 64, 16, lambda prob: None, n)
    dirty.sc[dirty.bt[1, 0], 0, 2, i] = what
    for uniform in (n, 0):
        out = attend(dirty, args, kind, uniform=uniform)
        assert torch.isnan(out[n:2 * n, 8:12]).all(), uniform
        out[n:2 * n, 8:12] = attend(clean, args, kind, uniform=uniform)[n:2 * n, 8:12]
        check(out, clean, f"uniform {uniform}")


# ------------------------------------------------------------------------------------------ keys that are not finite
@pytest.mark.parametrize("kind,n", [("decode", 1)] + [(k, n) for k in ("window", "tree") for n in (1, 4, 33, 90)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_a_key_that_is_not_finite_stays_with_its_sequence_and_head(kind, n, what, where):
    """A key that every query of a sequence sees: other sequences and kv heads are as without it, and a NaN reaches those
    who see it."""
    lens = [n + 30, 300 + n, 517]
    if kind != "tree":
        sees, args = [window_sees(L, n, 130, 20) for L in lens], (130, 20)
    else:
        masks = random_trees([n] * 3, 3, np.random.default_rng(n), noise=False)
        sees = [tree_sees(L, n, masks[b * n:b * n + n]) for b, L in enumerate(lens)]
        args = (torch.from_numpy(masks).cuda(),)
    prob = Problem("bf16", sees, 16, 4, 64, 32, seed=n)
    q, c, bt, ld, cu = prob.cuda()
    spoilt = [t.clone() for t in c]
    spoilt[where == "v"][bt[1, 0].item(), 7, 2, 5] = what
    for uniform in (n, 0) if kind != "decode" else (None,):
        give = lambda cache: (decode(prob, *args, dev=(q, cache, bt, ld, cu)) if kind == "decode" else
                              attend(prob, args, kind, uniform=uniform, dev=(q, cache, bt, ld, cu)))
        out = give(spoilt)
        hit = out[n:2 * n, 8:12]
        if what != what:
            assert torch.isnan(hit if where == "k" else hit[..., 5]).all()
        if where == "v":
            assert not torch.isfinite(hit[..., 5]).any()
        out[n:2 * n, 8:12] = give(c)[n:2 * n, 8:12]
        check(out, prob, f"uniform {uniform}", long_runs=True)


# ------------------------------------------------------------------------------------------ long tables
@pytest.mark.parametrize("cache,n", [("bf16", 1), ("fp8", 1), ("int8", 1), ("bf16", 3), ("int8", 3), ("bf16", 20),
                                     ("int8", 20)])
def test_short_windows_at_the_end_of_long_tables(cache, n):
    """256 sequences of up to 9.6 million tokens, of which a window's are there: the list has what is seen."""
    B, bs, mb = 256, 16, 600_000
    rng = np.random.default_rng(n)
    lens = [int(L) for L in rng.integers(n, 200, B)]
    prob = Problem(cache, [window_sees(L, n, 50, 0) for L in lens], 16, 8, 64, bs, seed=n)
    q, c, bt, ld, cu = prob.cuda()
    shift = torch.from_numpy(rng.integers(0, mb - bt.shape[1], B)).int().cuda()
    shift[0] = mb - bt.shape[1]
    shift[[b for b in range(B) if lens[b] < 50 + n]] = 0  # (their windows begin at the sequence's start)
    table = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    table.scatter_(1, (shift[:, None] + torch.arange(bt.shape[1], device="cuda")).long(), bt)
    dev = (q, c, table, ld + shift * bs, cu)
    if n == 1:
        check(decode(prob, 50, 0, dev=dev), prob, "decode")
    for uniform in (n, 0) if cache != "fp8" else ():
        check(attend(prob, (50, 0), uniform=uniform, dev=dev), prob, f"uniform {uniform}", long_runs=True)


# ------------------------------------------------------------------------------------------ the weights' precision
def one_part(prob):
    """The result with each softmax weight rounded to one bf16 part, the sum of weights taken before that (64 bits on
    the CPU)."""
    out, r, G = torch.zeros(prob.q.shape, dtype=torch.float64), 0, prob.Hq // prob.Hkv
    for b, s in enumerate(prob.sees):
        n, L = s.shape
        if n:
            at = torch.arange(L)
            page, row = torch.from_numpy(prob.bt[b].astype(np.int64))[at // prob.bs], at % prob.bs
            k, v = (torch.nan_to_num(t[page, row]) for t in (prob.kd, prob.vd))
            x = torch.einsum("nhgd,lhd->hgnl", prob.q[r:r + n].double().view(n, prob.Hkv, G, prob.D), k) * prob.scale
            x = x.masked_fill(torch.from_numpy(~s), float("-inf"))
            p = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.einsum("hgnl,lhd->nhgd", p.bfloat16().double(), v) / p.sum(-1).permute(2, 0, 1)[..., None]
            out[r:r + n] = o.reshape(n, prob.Hq, prob.D)
        r += n
    return out


@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("Hq,Hkv,D,bs,most", [(16, 8, 128, 16, 16), (8, 8, 64, 64, 32), (16, 2, 64, 256, 4),
                                              (15, 5, 128, 32, 10)])
def test_few_new_tokens_keep_their_weights(kind, Hq, Hkv, D, bs, most):
    """Up to twice the tokens of one pass on average, by offsets or all alike: the weights' parts are those of the plain
    attention of as many (2^-16), whichever way the call says how many there are."""
    rng = np.random.default_rng(most)
    for new in ([1] * 24, [1, 3, 2, 1] * 6, [most] * 6, [most + 3, 1, most - 1, most - 3]):
        lens = [n + int(rng.integers(1, 6)) for n in new]
        if kind == "window":
            sees, args = [window_sees(L, n, 5, 1) for L, n in zip(lens, new)], (5, 1)
        else:
            masks = random_trees(new, 2, rng, noise=False)
            cu = np.concatenate([[0], np.cumsum(new)])
            sees, args = [tree_sees(L, n, masks[a:a + n]) for L, n, a in zip(lens, new, cu)], None
        prob = Problem("bf16", sees, Hq, Hkv, D, bs, seed=len(new))
        want, mag = prob.want()
        over = (one_part(prob) - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -11 * mag)
        assert over.max() > 0  # one part would show
        args = args or (torch.from_numpy(masks).cuda(),)
        check(attend(prob, args, kind), prob, f"offsets, {new}")
        if len(set(new)) == 1:
            check(attend(prob, args, kind, uniform=new[0]), prob, f"uniform, {new}")
