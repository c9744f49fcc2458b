"""What the attention over the cache refuses for its size, before any device work."""
import pytest

from test_cache_abi import INVALID, UNSUPPORTED, _attend, _err, lib  # noqa: F401


@pytest.mark.parametrize("kw,text", [
    (dict(width=1 << 26, ts=1 << 26), "2^31 positions"),
    (dict(width=1 << 24, ts=1 << 24, n=1024, hq=64, hkv=8, q_hs=128), "too many"),      # 2^31 tiles of 128
    (dict(width=1 << 24, ts=1 << 24, n=1, hq=128, hkv=128), "too many"),                # 2^31 tiles of 64
])
def test_attend_refuses_tables_that_are_too_large(lib, kw, text):                       # noqa: F811
    assert _attend(lib, **kw) == UNSUPPORTED
    assert text in _err(lib)


@pytest.mark.parametrize("scale", [1.5e37, 3e38])
def test_attend_refuses_scales_that_overflow(lib, scale):                               # noqa: F811
    """16 scale log2 e has to be finite."""
    assert _attend(lib, scale=scale) == INVALID
    assert "scale > 0 and < 1.4e37" in _err(lib)
