"""GPU tests of windowed and tree calls at their edges: drafted nodes that nobody sees.  Bounds as in test_gpu_masks.py.
"""
import numpy as np
import pytest
import torch

from mask_reference import Problem, random_trees, tree_sees
from paged_kv_cache_62_gb300 import pkv
from test_gpu_masks import attend, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


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
