"""Refusals of the int8-cache and rotary entry points, on the host before any CUDA call (FAKE is never
dereferenced), and of their bindings."""
import pytest
import torch

from paged_kv_cache_62_gb300 import build as pkv_build
from paged_kv_cache_62_gb300 import pkv

NULL, FAKE = None, 0x10000


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load()


def swap(names, base, **kw):
    assert set(kw) <= set(names)
    return [kw.get(n, b) for n, b in zip(names, base)]


STORE = "k v ks vs bt mb cu lens B T n kc vc sc NB bs Hkv D err st".split()
STORE_OK = [FAKE, FAKE, 1024, 1024, FAKE, 4, FAKE, FAKE, 2, 5, 0, FAKE, FAKE, FAKE, 10, 16, 8, 128, NULL, NULL]


@pytest.mark.parametrize("kw,status", [
    (dict(k=NULL), pkv.EINVAL), (dict(v=FAKE + 8), pkv.EINVAL), (dict(cu=NULL), pkv.EINVAL),
    (dict(sc=NULL), pkv.EINVAL), (dict(sc=FAKE + 4), pkv.EINVAL), (dict(kc=FAKE + 8), pkv.EINVAL),
    (dict(ks=1016), pkv.EINVAL), (dict(vs=1028), pkv.EINVAL), (dict(n=2), pkv.EINVAL), (dict(T=-1), pkv.EINVAL),
    (dict(B=0), pkv.EINVAL), (dict(D=96), pkv.EUNSUPPORTED), (dict(bs=8), pkv.EUNSUPPORTED),
    (dict(bs=48), pkv.EUNSUPPORTED), (dict(bs=2048), pkv.EUNSUPPORTED), (dict(NB=1 << 28), pkv.EBOUNDS),
    (dict(T=0, k=NULL, cu=NULL), pkv.OK),
])
def test_store_i8(lib, kw, status):
    assert lib.pkv_kv_store_i8(*swap(STORE, STORE_OK, **kw)) == status


DEC = "q kc vc sc bt mb lens B Hq Hkv D bs NB mx scale out ws wsb workers err st".split()
DEC_OK = [FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, 2, 16, 8, 128, 16, 10, 64, 0.1, FAKE, FAKE, 1 << 30, 0, NULL, NULL]


@pytest.mark.parametrize("kw,status", [
    (dict(sc=NULL), pkv.EINVAL), (dict(sc=FAKE + 4), pkv.EINVAL), (dict(q=FAKE + 2), pkv.EINVAL),
    (dict(D=96), pkv.EUNSUPPORTED), (dict(Hq=136), pkv.EUNSUPPORTED), (dict(bs=8), pkv.EUNSUPPORTED),
    (dict(Hq=12), pkv.EINVAL), (dict(scale=float("inf")), pkv.EINVAL), (dict(wsb=64), pkv.EWORKSPACE),
    (dict(ws=NULL), pkv.EWORKSPACE), (dict(workers=pkv.MAX_WORKERS + 1), pkv.EBOUNDS),
    (dict(B=pkv.MAX_SEQS + 1), pkv.EBOUNDS), (dict(B=0, q=NULL), pkv.OK),
])
def test_decode_i8(lib, kw, status):
    assert lib.pkv_paged_decode_i8(*swap(DEC, DEC_OK, **kw)) == status


ATT = "q kc vc sc bt mb cu lens B T Hq Hkv D bs NB mx scale out n ws wsb workers err st".split()
ATT_OK = [FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, FAKE, 2, 5, 16, 8, 128, 16, 10, 64, 0.1, FAKE, 0, FAKE, 1 << 30, 0,
          NULL, NULL]


@pytest.mark.parametrize("kw,status", [
    (dict(cu=NULL), pkv.EINVAL), (dict(n=3), pkv.EINVAL), (dict(lens=NULL), pkv.EINVAL), (dict(B=0), pkv.EINVAL),
    (dict(T=pkv.MAX_SEQS + 1), pkv.EBOUNDS), (dict(wsb=64), pkv.EWORKSPACE), (dict(Hq=12), pkv.EINVAL),
    (dict(Hq=136), pkv.EUNSUPPORTED), (dict(Hq=4096, T=500), pkv.EUNSUPPORTED), (dict(D=96, T=500), pkv.EUNSUPPORTED),
    (dict(T=500, out=NULL), pkv.EINVAL), (dict(T=500, out=FAKE + 8), pkv.EINVAL), (dict(T=0, q=NULL), pkv.OK),
])
def test_attention_i8(lib, kw, status):
    assert lib.pkv_paged_attention_i8(*swap(ATT, ATT_OK, **kw)) == status


@pytest.mark.parametrize("T", [5, 30, 500])
@pytest.mark.parametrize("kw,status", [
    (dict(mx=-1), pkv.EINVAL), (dict(mb=0), pkv.EINVAL), (dict(NB=0), pkv.EINVAL), (dict(bs=0), pkv.EINVAL),
    (dict(workers=-1), pkv.EINVAL), (dict(scale=float("nan")), pkv.EINVAL), (dict(kc=NULL), pkv.EINVAL),
    (dict(sc=FAKE + 4), pkv.EINVAL), (dict(vc=FAKE + 8), pkv.EINVAL), (dict(bt=NULL), pkv.EINVAL),
    (dict(bs=8), pkv.EUNSUPPORTED), (dict(bs=48), pkv.EUNSUPPORTED), (dict(workers=1 << 20), pkv.EBOUNDS),
    (dict(NB=1 << 28), pkv.EBOUNDS),
])
def test_attention_i8_refuses_before_it_launches(lib, T, kw, status):
    assert lib.pkv_paged_attention_i8(*swap(ATT, ATT_OK, T=T, **kw)) == status


COPY = "kc vc sc pairs n NB bs Hkv D err st".split()
COPY_OK = [FAKE, FAKE, FAKE, FAKE, 3, 10, 16, 8, 128, NULL, NULL]


@pytest.mark.parametrize("kw,status", [
    (dict(sc=NULL), pkv.EINVAL), (dict(pairs=NULL), pkv.EINVAL), (dict(n=-1), pkv.EINVAL),
    (dict(bs=24), pkv.EUNSUPPORTED), (dict(vc=FAKE + 8), pkv.EINVAL), (dict(NB=1 << 30), pkv.EBOUNDS),
    (dict(n=0, kc=NULL), pkv.OK),
])
def test_copy_i8(lib, kw, status):
    assert lib.pkv_copy_blocks_i8(*swap(COPY, COPY_OK, **kw)) == status


ROPE = "q qs k ks pos axes inv ax T Hq Hkv D rot inter qo qos ko kos err st".split()
ROPE_OK = [FAKE, 2048, FAKE, 1024, FAKE, 3, FAKE, NULL, 5, 16, 8, 128, 128, 0, FAKE, 2048, FAKE, 1024, NULL, NULL]


@pytest.mark.parametrize("kw,status", [
    (dict(q=NULL), pkv.EINVAL), (dict(ko=NULL), pkv.EINVAL), (dict(pos=NULL), pkv.EINVAL), (dict(inv=NULL), pkv.EINVAL),
    (dict(qs=2040), pkv.EINVAL), (dict(kos=1020), pkv.EINVAL), (dict(ks=1026), pkv.EINVAL), (dict(axes=0), pkv.EINVAL),
    (dict(rot=144), pkv.EINVAL), (dict(rot=40), pkv.EUNSUPPORTED), (dict(D=136, qs=4096, qos=4096), pkv.EUNSUPPORTED),
    (dict(D=512, qs=1 << 14, qos=1 << 14, ks=1 << 14), pkv.EUNSUPPORTED), (dict(qo=FAKE + 8), pkv.EINVAL),
    (dict(T=-1), pkv.EINVAL), (dict(T=0, q=NULL), pkv.OK),
])
def test_rope(lib, kw, status):
    assert lib.pkv_rope(*swap(ROPE, ROPE_OK, **kw)) == status


RS = "q qs k ks v vs pos axes inv ax slots T Hq Hkv D rot inter qo qos kc vc NB bs err st".split()
RS_OK = [FAKE, 2048, FAKE, 1024, FAKE, 1024, FAKE, 1, FAKE, NULL, FAKE, 5, 16, 8, 128, 128, 0, FAKE, 2048, FAKE, FAKE,
         10, 16, NULL, NULL]


@pytest.mark.parametrize("kw,status", [
    (dict(v=NULL), pkv.EINVAL), (dict(vs=1000), pkv.EINVAL), (dict(slots=NULL), pkv.EINVAL), (dict(kc=NULL), pkv.EINVAL),
    (dict(vc=FAKE + 8), pkv.EINVAL), (dict(NB=0), pkv.EINVAL), (dict(T=0, v=NULL), pkv.OK),
])
def test_rope_store(lib, kw, status):
    assert lib.pkv_rope_store(*swap(RS, RS_OK, **kw)) == status


def test_bindings_refuse_cpu_tensors_and_bad_shapes(lib):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    kc, sc, i32 = z(4, 16, 2, 64, dt=torch.int8), z(4, 1, 2, 2, dt=torch.float32), torch.int32
    with pytest.raises(ValueError):
        pkv.kv_store_i8(z(2, 2, 64), z(2, 2, 64), kc, kc, sc, z(2, 3, dt=i32), z(2, dt=i32), new_per_seq=1)
    with pytest.raises(ValueError):
        pkv.paged_decode_i8(z(2, 4, 64), kc, kc, sc, z(2, 3, dt=i32), z(2, dt=i32), 0.1, z(2, 4, 64),
                            z(64, dt=torch.uint8))
    with pytest.raises(ValueError):
        pkv.copy_blocks_i8(kc, kc, sc, z(1, 2, dt=i32))
    with pytest.raises(ValueError):
        pkv.rope(z(2, 4, 64), z(2, 2, 64), z(2, dt=i32), z(32, dt=torch.float32), z(2, 4, 64), z(2, 2, 64))
    with pytest.raises(ValueError):
        pkv.alloc_i8_cache(4, 8, 2, 64)


# ------------------------------------------------------------------------------------------ workspaces
# bytes that bf16 calls of these sizes took before the library had int8 caches
BF16_SIZES = {(16384, 36, 4, 128): 42893568, (4096, 9, 1, 64): 19939584, (256, 16, 8, 128): 68324608,
              (1, 4, 2, 64): 17533952, (3000, 14, 2, 64): 30861824, (100, 15, 5, 128): 63314432,
              (60, 16, 1, 128): 38237184, (500, 20, 1, 64): 42917120}


@pytest.mark.parametrize("sizes", sorted(BF16_SIZES))
def test_bf16_attention_takes_the_workspace_it_took(lib, sizes):
    T, Hq, Hkv, D = sizes
    need = BF16_SIZES[sizes]
    assert lib.pkv_paged_attention_workspace_size(*sizes) == need
    assert lib.pkv_paged_attention_i8_workspace_size(*sizes) >= need
    names = [n for n in ATT if n != "sc"]
    base = [v for n, v in zip(ATT, ATT_OK) if n != "sc"]
    if Hq // Hkv <= 16:
        # a size it takes: the call goes on and ends at the device that is missing here
        kw = dict(T=T, Hq=Hq, Hkv=Hkv, D=D)
        assert lib.pkv_paged_attention(*swap(names, base, wsb=need - 1, **kw)) == pkv.EWORKSPACE
        assert lib.pkv_paged_attention_i8(*swap(ATT, ATT_OK, wsb=need - 1, **kw)) == pkv.EWORKSPACE
        if not torch.cuda.is_available():
            assert lib.pkv_paged_attention(*swap(names, base, wsb=need, **kw)) == pkv.ECUDA
            assert lib.pkv_paged_attention_i8(*swap(ATT, ATT_OK, wsb=need, **kw)) == pkv.ECUDA


def test_int8_attention_workspace_sizes(lib):
    f, g = lib.pkv_paged_attention_i8_workspace_size, lib.pkv_paged_attention_workspace_size
    assert f(0, 16, 8, 128) == g(0, 16, 8, 128) and f(-1, 16, 8, 128) == 0 and f(4, 16, 6, 128) == 0
    assert f(pkv.MAX_SEQS + 1, 16, 8, 128) == 0
    for rows in (1, 60, 500, pkv.MAX_SEQS):
        for hq, hkv, d in ((16, 8, 128), (14, 2, 64), (9, 1, 64), (16, 1, 128), (15, 5, 128)):
            assert f(rows, hq, hkv, d) >= g(rows, hq, hkv, d)
            assert f(rows, hq, hkv, d) <= f(rows + 100, hq, hkv, d) or rows + 100 > pkv.MAX_SEQS


# ------------------------------------------------------------------------------------------ long unit lists
def test_unit_lists_beyond_32_bits_are_refused_before_anything_is_launched(lib):
    """16000 rows of 100 sequences of up to 2^31 - 1 tokens: 350 entries x 8 kv heads x 2^24 tiles; the same in runs
    of a few rows (a launch would end in ECUDA here)."""
    kw = dict(mb=1 << 27, mx=(1 << 31) - 1)
    assert lib.pkv_paged_attention_i8(*swap(ATT, ATT_OK, T=16000, B=100, **kw)) == pkv.EBOUNDS
    assert lib.pkv_paged_attention_i8(*swap(ATT, ATT_OK, T=7000, B=7000, **kw)) == pkv.EBOUNDS
    assert lib.pkv_paged_decode_i8(*swap(DEC, DEC_OK, B=7000, **kw)) == pkv.EBOUNDS


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would go on to their launch")
def test_long_tables_are_not_refused(lib):
    """A list of at most 16384 x 4096 units (32 tokens of 8 kv heads) fits 32 bits by far."""
    kw = dict(B=pkv.MAX_SEQS, mb=8192, mx=131072)
    assert lib.pkv_paged_decode_i8(*swap(DEC, DEC_OK, **kw)) == pkv.ECUDA
    assert lib.pkv_paged_attention_i8(*swap(ATT, ATT_OK, D=64, T=pkv.MAX_SEQS, **kw)) == pkv.ECUDA


# ------------------------------------------------------------------------------------------ allocation
def test_an_int8_cache_has_fp32_scales_whatever_the_default_type():
    """Engines set the model's type as torch's default."""
    old = torch.get_default_dtype()
    torch.set_default_dtype(torch.bfloat16)
    try:
        k, v, sc = pkv.alloc_i8_cache(3, 32, 2, 64, device="cpu")
    finally:
        torch.set_default_dtype(old)
    assert k.dtype == v.dtype == torch.int8 and sc.dtype == torch.float32
    assert k.shape == v.shape == (3, 32, 2, 64) and sc.shape == (3, 2, 2, 2)


@pytest.mark.parametrize("alloc,args", [(pkv.alloc_i8_cache, (3, 32, 2, 64)), (pkv.alloc_workspace, (2, 4, 2, 64)),
                                        (pkv.alloc_attention_workspace, (5, 4, 2, 64))])
def test_device_0_is_a_device(lib, monkeypatch, alloc, args):
    """Device index 0 is not taken as "none given" (the current device)."""
    asked = []
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **kw: asked.append(device) or zeros(*a, **kw))
    alloc(*args, device=0)
    assert asked and all(d == 0 and d is not None and not isinstance(d, str) for d in asked)
    asked.clear()
    alloc(*args)
    assert asked and all(d == "cuda" for d in asked)
