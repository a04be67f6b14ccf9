"""Refusals of the windowed, tree and normed rotary entry points, on the host before any CUDA call (FAKE is never
dereferenced)."""
import pytest

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


CACHES = {"": [], "_fp8": ["ks", "vs"], "_i8": ["sc"]}


def decode(lib, kind, **kw):
    names = "q kc vc".split() + CACHES[kind] + "bt mb lens B Hq Hkv D bs NB mx scale w s out ws wsb workers err st".split()
    base = [FAKE] * (3 + len(CACHES[kind])) + [FAKE, 4, FAKE, 2, 16, 8, 128, 16, 10, 64, 0.1, 32, 4, FAKE, FAKE, 1 << 30,
                                               0, NULL, NULL]
    return getattr(lib, f"pkv_paged_decode_window{kind}")(*swap(names, base, **kw))


@pytest.mark.parametrize("kind", list(CACHES))
@pytest.mark.parametrize("kw,status", [
    (dict(w=0), pkv.EINVAL), (dict(w=-5), pkv.EINVAL), (dict(s=-1), pkv.EINVAL), (dict(q=FAKE + 2), pkv.EINVAL),
    (dict(kc=NULL), pkv.EINVAL), (dict(D=96), pkv.EUNSUPPORTED), (dict(Hq=136), pkv.EUNSUPPORTED),
    (dict(bs=48), pkv.EUNSUPPORTED), (dict(Hq=12), pkv.EINVAL), (dict(scale=float("inf")), pkv.EINVAL),
    (dict(wsb=64), pkv.EWORKSPACE), (dict(ws=NULL), pkv.EWORKSPACE), (dict(workers=pkv.MAX_WORKERS + 1), pkv.EBOUNDS),
    (dict(B=pkv.MAX_SEQS + 1), pkv.EBOUNDS), (dict(mb=1 << 27, mx=(1 << 30) + 1, Hkv=1, Hq=1, B=1), pkv.EBOUNDS),
    (dict(B=0, q=NULL), pkv.OK), (dict(B=0, w=0), pkv.EINVAL),
])
def test_decode_window(lib, kind, kw, status):
    assert decode(lib, kind, **kw) == status


def test_decode_window_scales(lib):
    assert decode(lib, "_fp8", ks=NULL) == pkv.EINVAL
    assert decode(lib, "_i8", sc=FAKE + 4) == pkv.EINVAL
    assert decode(lib, "_i8", bs=8) == pkv.EUNSUPPORTED


def attention(lib, kind, cache, **kw):
    mask = ["w", "s"] if kind == "window" else ["mask", "words"]
    names = "q kc vc".split() + CACHES[cache] + "bt mb cu lens B T Hq Hkv D bs NB mx scale".split() + mask + \
        "out n ws wsb workers err st".split()
    base = [FAKE] * (3 + len(CACHES[cache])) + [FAKE, 4, FAKE, FAKE, 2, 5, 16, 8, 128, 16, 10, 64, 0.1] + \
        ([32, 4] if kind == "window" else [FAKE, 2]) + [FAKE, 0, FAKE, 1 << 30, 0, NULL, NULL]
    return getattr(lib, f"pkv_paged_attention_{kind}{cache}")(*swap(names, base, **kw))


@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("cache", ["", "_i8"])
@pytest.mark.parametrize("T", [5, 30, 500])
@pytest.mark.parametrize("kw,status", [
    (dict(cu=NULL), pkv.EINVAL), (dict(n=3), pkv.EINVAL), (dict(lens=NULL), pkv.EINVAL), (dict(B=0), pkv.EINVAL),
    (dict(wsb=64), pkv.EWORKSPACE), (dict(Hq=12), pkv.EINVAL), (dict(Hq=136), pkv.EUNSUPPORTED),
    (dict(D=96), pkv.EUNSUPPORTED), (dict(out=NULL), pkv.EINVAL), (dict(out=FAKE + 8), pkv.EINVAL),
    (dict(mx=-1), pkv.EINVAL), (dict(mb=0), pkv.EINVAL), (dict(NB=0), pkv.EINVAL), (dict(bs=0), pkv.EINVAL),
    (dict(workers=-1), pkv.EINVAL), (dict(scale=float("nan")), pkv.EINVAL), (dict(kc=NULL), pkv.EINVAL),
    (dict(vc=FAKE + 8), pkv.EINVAL), (dict(bt=NULL), pkv.EINVAL), (dict(bs=48), pkv.EUNSUPPORTED),
    (dict(workers=1 << 20), pkv.EBOUNDS), (dict(NB=1 << 28), pkv.EBOUNDS),
    (dict(mb=1 << 27, mx=(1 << 30) + 1, Hkv=1, Hq=1), pkv.EBOUNDS),
])
def test_attention_refuses_before_it_launches(lib, kind, cache, T, kw, status):
    assert attention(lib, kind, cache, T=T, **kw) == status


@pytest.mark.parametrize("cache", ["", "_i8"])
def test_attention_masks(lib, cache):
    for kw in (dict(w=0), dict(s=-1), dict(w=-1, T=0)):
        assert attention(lib, "window", cache, **kw) == pkv.EINVAL
    for kw in (dict(mask=NULL), dict(mask=FAKE + 2), dict(words=0), dict(words=-1), dict(B=2, T=130, n=65),
               dict(B=2, T=66, n=33, words=1)):
        assert attention(lib, "tree", cache, **kw) == pkv.EINVAL
    assert attention(lib, "tree", cache, T=0, mask=NULL) == pkv.OK
    assert attention(lib, "window", cache, T=pkv.MAX_SEQS + 1) == pkv.EBOUNDS


ROPE = "q qs k ks qw kw eps pos axes inv ax T Hq Hkv D rot inter qo qos ko kos err st".split()
ROPE_OK = [FAKE, 2048, FAKE, 1024, FAKE, FAKE, 1e-6, FAKE, 3, FAKE, NULL, 5, 16, 8, 128, 128, 0, FAKE, 2048, FAKE, 1024,
           NULL, NULL]
RS = "q qs k ks v vs qw kw eps pos axes inv ax slots T Hq Hkv D rot inter qo qos kc vc NB bs err st".split()
RS_OK = [FAKE, 2048, FAKE, 1024, FAKE, 1024, FAKE, FAKE, 1e-6, FAKE, 1, FAKE, NULL, FAKE, 5, 16, 8, 128, 128, 0, FAKE,
         2048, FAKE, FAKE, 10, 16, NULL, NULL]
NORM = [(dict(eps=0.0), pkv.EINVAL), (dict(eps=-1e-6), pkv.EINVAL), (dict(eps=float("nan")), pkv.EINVAL),
        (dict(eps=float("inf")), pkv.EINVAL), (dict(qw=FAKE + 4), pkv.EINVAL), (dict(kw=FAKE + 8), pkv.EINVAL),
        (dict(q=NULL), pkv.EINVAL), (dict(pos=NULL), pkv.EINVAL), (dict(qs=2040), pkv.EINVAL),
        (dict(rot=144), pkv.EINVAL), (dict(rot=40), pkv.EUNSUPPORTED), (dict(T=-1), pkv.EINVAL),
        (dict(T=0, q=NULL), pkv.OK), (dict(T=0, eps=0.0), pkv.EINVAL)]


@pytest.mark.parametrize("kw,status", NORM)
def test_qk_norm_rope(lib, kw, status):
    assert lib.pkv_qk_norm_rope(*swap(ROPE, ROPE_OK, **kw)) == status


@pytest.mark.parametrize("kw,status", NORM + [(dict(v=NULL), pkv.EINVAL), (dict(slots=NULL), pkv.EINVAL),
                                              (dict(vc=FAKE + 8), pkv.EINVAL), (dict(NB=0), pkv.EINVAL)])
def test_qk_norm_rope_store(lib, kw, status):
    assert lib.pkv_qk_norm_rope_store(*swap(RS, RS_OK, **kw)) == status
