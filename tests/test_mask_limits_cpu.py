"""The limit on a masked call's unit list counts what its queries see, not the table's length: checked on the host before
any CUDA call (FAKE is never dereferenced)."""
import pytest
import torch

from paged_kv_cache_62_gb300 import build as pkv_build
from paged_kv_cache_62_gb300 import pkv
from test_masks_norm_cpu import attention, decode


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load()


LONG = dict(B=256, mb=1 << 25, mx=1 << 29)  # 2^29 tokens a table of pages of 16, 256 sequences of 8 kv heads


@pytest.mark.parametrize("kind", ["", "_fp8", "_i8"])
def test_decode_windows_over_long_tables(lib, kind):
    """A short window passes this check (the next one refuses the workspace), one as long as the table does not."""
    for window in (1, 32, 4096):
        assert decode(lib, kind, w=window, s=16, ws=None, **LONG) == pkv.EWORKSPACE
    assert decode(lib, kind, w=1 << 29, ws=None, **LONG) == pkv.EBOUNDS
    assert decode(lib, kind, w=1, s=1 << 29, ws=None, **LONG) == pkv.EBOUNDS


@pytest.mark.skipif(torch.cuda.is_available(), reason="the arguments pass every check")
@pytest.mark.parametrize("cache", ["", "_i8"])
@pytest.mark.parametrize("n", [1, 2, 60])
def test_attention_windows_over_long_tables(lib, cache, n):
    T = 256 * n
    assert attention(lib, "window", cache, w=64, s=4, n=n, T=T, **LONG) == pkv.ECUDA  # (no device here)
    assert attention(lib, "window", cache, w=1 << 29, n=n, T=T, **LONG) == pkv.EBOUNDS
    assert attention(lib, "tree", cache, n=n, T=T, **LONG) == pkv.EBOUNDS
