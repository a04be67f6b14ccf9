"""GPU tests of the rotary positions and their fused store against a 64-bit reference.

Tolerance: the result rounds to bf16 by at most 2^-8 of itself; its two products, their sum and the cosine and
sine are fp32 (the angle is exact to 2^-24 turns' fraction and sincospif to 2 ulp), together at most
2^-20 (|x| + |y|) of the pair's elements.
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
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:]
    parts = [t.view(T, -1, D) for t in (q, k, v)]
    return parts if wide else [t.contiguous() for t in parts]


def close(got, x, pos, inv, axis_of, inter, what):
    want = rope64(x.cpu(), pos, inv, axis_of, inter)
    off = (got.cpu().double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -20 * 2 * x.abs().max().item())
    assert off.max() <= 0, f"{what}: over by {off.max():.3g}"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [(1, 16, 8, 128, 128), (37, 14, 2, 64, 64), (64, 4, 2, 64, 32),
                                            (5, 3, 1, 96, 48), (130, 32, 8, 128, 64), (3, 2, 2, 256, 256),
                                            (9, 1, 1, 16, 16), (17, 40, 40, 80, 80)])
def test_rope_one_axis(T, Hq, Hkv, D, rot, inter):
    q, k, _ = inputs(T, Hq, Hkv, D, T + rot)
    inv = freqs(rot)
    pos = np.arange(T)[None] * 37 + 5
    qo, ko = (torch.full(t.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for t in (q, k))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.rope(q, k, torch.tensor(pos[0], dtype=torch.int32, device="cuda"), torch.from_numpy(inv).cuda(), qo, ko,
             interleaved=inter, err_word=err)
    assert err.item() == 0
    zero = np.zeros(rot // 2, int)
    close(qo, q, pos, inv, zero, inter, "q")
    close(ko, k, pos, inv, zero, inter, "k")
    assert torch.equal(qo[..., rot:], q[..., rot:])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_rope_store_axes_and_slots(axes, inter):
    T, Hq, Hkv, D, bs, NB = 200, 16, 8, 128, 16, 20
    rng = np.random.default_rng(axes)
    q, k, v = inputs(T, Hq, Hkv, D, axes)
    inv = freqs(D)
    pos = rng.integers(0, 4000, (axes, T))
    axis_of = rng.integers(0, axes, D // 2)                   # any assignment, contiguous or woven
    slots = rng.permutation(NB * bs)[:T]
    slots[3] = slots[77] = -1
    kc, vc = (torch.full((NB, bs, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    pkv.rope_store(q, k, v, i32(pos), torch.from_numpy(inv).cuda(), i32(slots), qo, kc, vc, freq_axis=i32(axis_of),
                   interleaved=inter, err_word=err)
    assert err.item() == 0
    close(qo, q, pos, inv, axis_of, inter, "q")
    keep = torch.from_numpy(slots >= 0).cuda()
    at = torch.from_numpy(slots[slots >= 0].astype(np.int64)).cuda()
    kept = slots >= 0
    close(kc.view(-1, Hkv, D)[at], k[keep], pos[:, kept], inv, axis_of, inter, "k")
    assert torch.equal(vc.view(-1, Hkv, D)[at], v[keep])
    rest = torch.ones(NB * bs, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.all(kc.view(-1, Hkv, D)[rest] == 7.0) and torch.all(vc.view(-1, Hkv, D)[rest] == 7.0)


def test_far_and_negative_positions():
    """Whole turns cost no precision: positions to the ends of int32, frequencies from 1e-9 to 50."""
    T, D = 8, 64
    q, k, _ = inputs(T, 4, 1, D, 8)
    pos = np.array([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 1 << 20, -77777777]])
    for inv in (freqs(D), freqs(D, 1e4), np.geomspace(1e-9, 50.0, D // 2).astype(np.float32),
                -freqs(D), np.where(np.arange(D // 2) % 3 == 0, 0, 1e-30).astype(np.float32)):
        qo, ko = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(k.shape, dtype=k.dtype, device="cuda")
        pkv.rope(q, k, torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.from_numpy(inv).cuda(), qo, ko)
        close(qo, q, pos, inv, np.zeros(D // 2, int), False, "q")
        close(ko, k, pos, inv, np.zeros(D // 2, int), False, "k")


@pytest.mark.parametrize("inter", [False, True])
def test_rope_in_place(inter):
    T, Hq, Hkv, D = 33, 8, 4, 128
    q, k, _ = inputs(T, Hq, Hkv, D, 1)
    inv, pos = torch.from_numpy(freqs(D)).cuda(), torch.arange(T, dtype=torch.int32, device="cuda")
    qo, ko = (torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k))
    pkv.rope(q, k, pos, inv, qo, ko, interleaved=inter)
    pkv.rope(q, k, pos, inv, q, k, interleaved=inter)         # parts of one projection's rows, in place
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_bad_slots_and_axes_are_flagged():
    T, Hq, Hkv, D, bs, NB = 4, 2, 1, 64, 16, 2
    q, k, v = inputs(T, Hq, Hkv, D, 2)
    inv, pos = torch.from_numpy(freqs(D)).cuda(), torch.zeros(2, T, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(NB, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([NB * bs, -2, 5, -1], dtype=torch.int32, device="cuda")
    pkv.rope_store(q, k, v, pos, inv, slots, qo, kc, vc, err_word=err)
    assert err.item() == pkv.ERR_SLOT_RANGE
    assert torch.equal(qo, q) and torch.equal(vc.view(-1, Hkv, D)[5], v[2])
    assert torch.all(vc.view(-1, Hkv, D)[torch.arange(NB * bs) != 5] == 0)
    err.zero_()
    axis = torch.zeros(D // 2, dtype=torch.int32, device="cuda")
    axis[3] = 2
    pkv.rope_store(q, k, v, pos, inv, slots.clamp(-1, 5), qo, kc, vc, freq_axis=axis, err_word=err)
    assert err.item() == pkv.ERR_AXIS_RANGE


def test_captured_rope_store_replays():
    T, Hq, Hkv, D, bs, NB = 3, 16, 8, 128, 16, 4
    q, k, v = inputs(T, Hq, Hkv, D, 5, wide=False)
    inv = freqs(D)
    pos, slots = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
    slots.copy_(torch.tensor([-1, -1, -1], dtype=torch.int32))
    kc, vc = (torch.zeros(NB, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo = torch.empty_like(q)
    invd = torch.from_numpy(inv).cuda()
    call = lambda: pkv.rope_store(q, k, v, pos, invd, slots, qo, kc, vc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for p, s in (([0, 1, 2], [5, 6, 40]), ([9, 77, 3], [-1, 63, 0])):
        pos.copy_(torch.tensor(p, dtype=torch.int32))
        slots.copy_(torch.tensor(s, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        close(qo, q, np.array([p]), inv, np.zeros(D // 2, int), False, "q")
        at = [i for i in range(T) if s[i] >= 0]
        rows = [s[i] for i in at]
        close(kc.view(-1, Hkv, D)[rows], k[at], np.array([[p[i] for i in at]]), inv, np.zeros(D // 2, int), False, "k")
        assert torch.equal(vc.view(-1, Hkv, D)[rows], v[at])


def test_an_error_of_the_interleaved_argument_is_passed_on():
    class Neither:
        def __bool__(self):
            raise OverflowError("neither")

    q, k, v = inputs(2, 2, 1, 64, 0)
    qo, ko = torch.zeros(q.shape, dtype=q.dtype, device="cuda"), torch.zeros(k.shape, dtype=k.dtype, device="cuda")
    pos, inv = torch.ones(2, dtype=torch.int32, device="cuda"), torch.from_numpy(freqs(64)).cuda()
    with pytest.raises(OverflowError, match="neither"):
        pkv.rope(q, k, pos, inv, qo, ko, interleaved=Neither())
    assert not qo.any() and not ko.any()
