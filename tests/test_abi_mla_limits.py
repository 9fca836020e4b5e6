"""rda_mla_decode at the largest sizes (CPU): what a launch cannot hold is
refused before anything reaches a device."""
import pytest

from test_abi_mla import DECODE, SHAPE, WS, call, lib  # noqa: F401


@pytest.mark.parametrize("want,kw", [
    # the joining kernel has a wave per query row, four a workgroup, and one
    # launch holds fewer than 2^24 workgroups
    (SHAPE, dict(batch=1 << 14, tokens=64, heads=64)),
    (SHAPE, dict(batch=1, tokens=4, heads=1 << 24)),
    (SHAPE, dict(batch=(1 << 26) - 3, tokens=1, heads=1)),
    (WS, dict(batch=(1 << 26) - 4, tokens=1, heads=1, width=1)),
    (WS, dict(batch=(1 << 14) - 1, tokens=64, heads=64)),
])
def test_query_rows(lib, want, kw):  # noqa: F811
    assert call(lib.rda_mla_decode, DECODE, **dict(dict(ws_bytes=1000), **kw)) == want


@pytest.mark.parametrize("want,kw", [
    # row numbers are 32 bits, and tiles are fetched up to nine ahead of the last
    (SHAPE, dict(page_tokens=8, page_stride=8 * 576, width=(1 << 28) - 1)),
    (SHAPE, dict(page_tokens=64, width=(1 << 25) - 1)),
    (SHAPE, dict(page_tokens=512, page_stride=512 * 576, width=(1 << 22) - 1)),
    (WS, dict(page_tokens=8, page_stride=8 * 576, width=(1 << 28) - 128)),
    (WS, dict(page_tokens=1 << 16, page_stride=(1 << 16) * 576, width=(1 << 15) - 1)),
])
def test_cached_rows(lib, want, kw):  # noqa: F811
    assert call(lib.rda_mla_decode, DECODE, **dict(dict(batch=1, ws_bytes=1000), **kw)) == want
