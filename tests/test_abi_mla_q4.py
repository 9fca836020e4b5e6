"""The entry points of the 4-bit latent cache on the CPU: bad arguments are
refused with the documented status before anything reaches a device, and the
binding's own checks."""
import os

import pytest
import torch

from gated_delta_amd import rda
from test_abi_mla import (ALIAS, ALIGN, APPEND, DECODE, INF, NAN, NULL, OK, SHAPE, UNSUP, VALUE, WS, GiB, P,  # noqa: F401
                          call, lib)

DECODE = dict(DECODE, page_stride=64 * 400)
APPEND = dict(APPEND, page_stride=64 * 400)
READ = dict(cache=P + 4 * GiB, page_stride=64 * 400, num_pages=10, page_tokens=64, table=P + 3 * GiB, width=4,
            kv_lens=P + 2 * GiB, cu=P + GiB, num_seqs=2, total=3, out=P, out_stride=576, stream=None)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(batch=0)), (OK, dict(tokens=0)), (SHAPE, dict(batch=-1)), (SHAPE, dict(tokens=-1)),
    (SHAPE, dict(tokens=65)), (SHAPE, dict(heads=0)), (SHAPE, dict(prefix_len=-1)),
    (SHAPE, dict(batch=1 << 22, heads=1 << 10)), (SHAPE, dict(tokens=64, heads=1 << 20)),
    (SHAPE, dict(num_pages=-1)), (SHAPE, dict(width=-1)), (SHAPE, dict(page_tokens=0)),
    (UNSUP, dict(page_tokens=4)), (UNSUP, dict(page_tokens=48)), (UNSUP, dict(page_tokens=1 << 17)),
    (SHAPE, dict(page_stride=64 * 400 - 16)), (SHAPE, dict(page_stride=64 * 400 + 8)),
    (SHAPE, dict(page_stride=(1 << 40) + 16)), (SHAPE, dict(num_pages=0, prefix_len=5)),
    (VALUE, dict(scale=0.0)), (VALUE, dict(scale=-1.0)), (VALUE, dict(scale=NAN)), (VALUE, dict(scale=INF)),
    (NULL, dict(q=None)), (NULL, dict(o=None)), (NULL, dict(kv_lens=None)), (NULL, dict(table=None)),
    (NULL, dict(cache=None)), (NULL, dict(prefix_len=5)),
    (ALIGN, dict(q=P + 8)), (ALIGN, dict(cache=P + GiB + 8)), (ALIGN, dict(o=P + 4 * GiB + 2)),
    (ALIGN, dict(kv_lens=P + 3 * GiB + 2)), (ALIGN, dict(table=P + 2 * GiB + 1)), (ALIGN, dict(lse=P + 6 * GiB + 2)),
    (ALIGN, dict(ws=P + 5 * GiB + 8)), (WS, dict(ws=None)), (WS, dict(ws_bytes=1000)),
    (ALIAS, dict(o=P)), (ALIAS, dict(o=P + GiB)), (ALIAS, dict(lse=P + 4 * GiB)),
    (ALIAS, dict(o=P + GiB + 10 * 64 * 400 - 16)), (ALIAS, dict(ws=P + GiB)), (ALIAS, dict(o=P + 5 * GiB + 256)),
    (ALIAS, dict(lse=P + 3 * GiB)), (ALIAS, dict(prefix_table=P + 4 * GiB, prefix_len=5)),
])
def test_decode_refusals(lib, want, kw):  # noqa: F811
    assert call(lib.rda_mla_decode_q4, DECODE, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(batch=1 << 14, tokens=64, heads=64)), (SHAPE, dict(batch=1, tokens=4, heads=1 << 24)),
    (WS, dict(batch=(1 << 14) - 1, tokens=64, heads=64)),
    # row numbers are 32 bits, up to 72 tiles behind the last
    (SHAPE, dict(batch=1, page_tokens=8, page_stride=8 * 400, width=(1 << 28) - 1)),
    (SHAPE, dict(batch=1, page_tokens=8, page_stride=8 * 400, width=(1 << 28) - 511)),
    (WS, dict(batch=1, page_tokens=8, page_stride=8 * 400, width=(1 << 28) - 512)),
    # and so are the places of the line that is cut into shares: a sequence's
    # tiles and six more for each 32 query rows
    (WS, dict(batch=1 << 25, heads=1, width=2)), (WS, dict(batch=1 << 25, heads=1, width=28)),
    (SHAPE, dict(batch=1 << 25, heads=1, width=30)),
    (SHAPE, dict(batch=1 << 25, heads=1, page_tokens=1 << 10, page_stride=400 << 10, width=2)),
])
def test_decode_limits(lib, want, kw):  # noqa: F811
    assert call(lib.rda_mla_decode_q4, DECODE, **dict(dict(ws_bytes=1000), **kw)) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(total=0)), (SHAPE, dict(num_seqs=0)), (SHAPE, dict(total=-1)), (SHAPE, dict(cu=None)),
    (OK, dict(cu=None, total=0)), (SHAPE, dict(kv_stride=568)), (SHAPE, dict(kv_stride=580)),
    (SHAPE, dict(kv_stride=(1 << 24) + 8)), (SHAPE, dict(total=(1 << 25) + 1)),
    (UNSUP, dict(page_tokens=12)), (SHAPE, dict(page_stride=100)), (SHAPE, dict(page_stride=64 * 400 + 8)),
    (VALUE, dict(eps=-1.0)), (VALUE, dict(eps=NAN)), (VALUE, dict(eps=INF)),
    (NULL, dict(kv=None)), (NULL, dict(kv_lens=None)), (NULL, dict(table=None)), (NULL, dict(cache=None)),
    (ALIGN, dict(kv=P + 2)), (ALIGN, dict(weight=P + 5 * GiB + 4)), (ALIGN, dict(cache=P + 4 * GiB + 8)),
    (ALIGN, dict(table=P + 3 * GiB + 1)), (ALIGN, dict(cu=P + GiB + 2)),
    (ALIAS, dict(cache=P)), (ALIAS, dict(kv_lens=P + 4 * GiB)), (ALIAS, dict(weight=P + 4 * GiB + 64)),
    (OK, dict(num_pages=0, cache=None)), (OK, dict(width=0, table=None)),
])
def test_append_refusals(lib, want, kw):  # noqa: F811
    assert call(lib.rda_mla_append_q4, APPEND, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(total=0)), (SHAPE, dict(num_seqs=0)), (SHAPE, dict(total=-1)), (SHAPE, dict(cu=None)),
    (OK, dict(cu=None, total=0)), (SHAPE, dict(out_stride=568)), (SHAPE, dict(out_stride=580)),
    (SHAPE, dict(total=(1 << 25) + 1)), (UNSUP, dict(page_tokens=12)), (SHAPE, dict(page_stride=100)),
    (NULL, dict(out=None)), (NULL, dict(kv_lens=None)), (NULL, dict(table=None)), (NULL, dict(cache=None)),
    (ALIGN, dict(out=P + 2)), (ALIGN, dict(cache=P + 4 * GiB + 8)), (ALIGN, dict(kv_lens=P + 2 * GiB + 1)),
    (ALIAS, dict(out=P + 4 * GiB)), (ALIAS, dict(out=P + 2 * GiB)), (ALIAS, dict(out=P + 3 * GiB)),
    (ALIAS, dict(cu=P)),
])
def test_read_refusals(lib, want, kw):  # noqa: F811
    assert call(lib.rda_mla_read_q4, READ, **kw) == want


def test_workspace_sizes(lib):  # noqa: F811
    W = rda.rda_mla_decode_q4_workspace_bytes
    assert W(0, 1, 32) > 0 and W(-1, 1, 32) == 0 and W(1, 65, 32) == 0 and W(1, 1, 0) == 0
    assert W(4, 1, 32, -1) == 0
    assert W(256, 3, 32) >= 256 * 96 * 512 * 4      # partial sums of every query row, fp32
    assert W(8, 1, 32, 100) >= W(8, 1, 32) + 8 * 32 * 512 * 4
    assert W(1 << 14, 64, 64) > (1 << 26) * 512 * 4


def test_constants_match_header():
    text = open(os.path.join(os.path.dirname(rda.library_path()), "..", "include", "rda.h")).read()
    assert f"#define RDA_MLA_ROW_Q4 {rda.RDA_MLA_ROW_Q4} " in text


def test_binding_refuses():
    """CPU tensors, other types, row widths and shapes that do not belong together."""
    i32 = dict(dtype=torch.int32)
    q, kv = torch.zeros(1, 1, 2, 576, dtype=torch.bfloat16), torch.zeros(3, 576, dtype=torch.bfloat16)
    cache, table, lens = torch.zeros(2, 8, 400, dtype=torch.uint8), torch.zeros(1, 1, **i32), torch.zeros(1, **i32)
    with pytest.raises(ValueError):
        rda.rda_mla_decode_q4(q, cache, table, lens, 1.0)
    with pytest.raises(ValueError):
        rda.rda_mla_append_q4(kv, cache, table, lens)
    with pytest.raises(ValueError):
        rda.rda_mla_read_q4(cache, table, lens, 3)
    with pytest.raises(TypeError):
        rda.rda_mla_append_q4(None, None, None, None)
    cpu = cache.device
    with pytest.raises(TypeError):
        rda._need_cache_q4(cache.to(torch.int8), cpu)
    for bad in (cache[..., :384], cache[0], cache[:, :, ::2], cache.transpose(0, 1), torch.zeros(2, 8, 576, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            rda._need_cache_q4(bad, cpu)
    # pages may lie apart
    wide = torch.zeros(2, 10, 400, dtype=torch.uint8)
    rda._need_cache_q4(wide[:, :8], cpu)
