"""The latent-attention and draft-verification entry points on the CPU: bad
arguments are refused with the documented status before anything reaches a
device, and the binding's own checks."""
import ctypes
import os

import pytest
import torch

from gated_delta_amd import rda

OK, NULL, SHAPE, UNSUP, DTYPE, WS, ALIGN, HIPERR, ALIAS, VALUE, TOO_LARGE = range(11)
P = 1 << 40          # fake, well-aligned device addresses: never dereferenced
GiB = 1 << 30
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(rda.library_path()):
        import gated_delta_amd.build as b
        b.build()
    return rda.lib()


def call(fn, defaults, **kw):
    unknown = set(kw) - set(defaults)
    assert not unknown, unknown
    return fn(*{**defaults, **kw}.values())


PREFILL = dict(q=P, q_stride=2 * 192, kv=P + GiB, kv_stride=2 * 256, k_pe=P + 2 * GiB, pe_stride=576,
               cu_q=P + 3 * GiB, cu_k=P + 4 * GiB, num_seqs=2, total_q=0, total_k=100, heads=2,
               scale=0.1, causal=1, o=P + 5 * GiB, lse=None, stream=None)
DECODE = dict(q=P, cache=P + GiB, page_stride=64 * 576, num_pages=10, page_tokens=64,
              table=P + 2 * GiB, width=4, kv_lens=P + 3 * GiB, prefix_table=None, prefix_len=0,
              batch=2, tokens=1, heads=32, scale=0.1, o=P + 4 * GiB, lse=None, ws=P + 5 * GiB,
              ws_bytes=GiB, stream=None)
APPEND = dict(kv=P, kv_stride=576, weight=None, eps=1e-5, cu=P + GiB, num_seqs=2, total=3,
              kv_lens=P + 2 * GiB, table=P + 3 * GiB, width=4, cache=P + 4 * GiB,
              page_stride=64 * 576, num_pages=10, page_tokens=64, stream=None)
VERIFY = dict(target=P, target_stride=1000, draft=P + GiB, draft_stride=1000, tokens=P + 2 * GiB,
              uniforms=P + 3 * GiB, num=None, batch=2, drafts=2, vocab=1000, accept=P + 4 * GiB,
              out=P + 5 * GiB, ws=P + 6 * GiB, ws_bytes=GiB, stream=None)


@pytest.mark.parametrize("want,kw", [
    (OK, {}), (SHAPE, dict(num_seqs=0)), (SHAPE, dict(total_q=-1)), (SHAPE, dict(total_k=-1)),
    (SHAPE, dict(heads=0)), (SHAPE, dict(cu_q=None)), (SHAPE, dict(cu_q=None, cu_k=None)),
    (SHAPE, dict(cu_k=None)), (OK, dict(cu_k=None, total_k=0)),
    (OK, dict(cu_q=None, cu_k=None, num_seqs=1)),
    (SHAPE, dict(q_stride=383)), (SHAPE, dict(q_stride=376)), (SHAPE, dict(kv_stride=508)),
    (SHAPE, dict(kv_stride=(1 << 24) + 8)), (SHAPE, dict(pe_stride=56)),
    (SHAPE, dict(heads=1 << 20, total_q=1 << 30)), (SHAPE, dict(heads=40000, q_stride=40000 * 192, kv_stride=40000 * 256, total_q=1 << 30)),
    (VALUE, dict(scale=0.0)), (VALUE, dict(scale=-1.0)), (VALUE, dict(scale=NAN)),
    (VALUE, dict(scale=INF)), (VALUE, dict(causal=2)), (VALUE, dict(causal=-1)),
    (NULL, dict(total_q=5, q=None)), (NULL, dict(total_q=5, o=None)), (NULL, dict(total_q=5, kv=None)),
    (NULL, dict(total_q=5, k_pe=None)),
    (ALIGN, dict(total_q=5, q=P + 8)), (ALIGN, dict(total_q=5, kv=P + GiB + 2)),
    (ALIGN, dict(total_q=5, k_pe=P + 4)), (ALIGN, dict(total_q=5, o=P + 5 * GiB + 8)),
    (ALIGN, dict(total_q=5, lse=P + 6 * GiB + 2)), (ALIGN, dict(total_q=5, cu_q=P + 3 * GiB + 1)),
    (ALIAS, dict(total_q=5, o=P)), (ALIAS, dict(total_q=5, o=P + GiB + 512)),
    (ALIAS, dict(total_q=5, lse=P + 5 * GiB)), (ALIAS, dict(total_q=5, lse=P + 2 * GiB)),
    (ALIAS, dict(total_q=5, o=P + 4 * GiB)),
])
def test_prefill_refusals(lib, want, kw):
    assert call(lib.rda_mla_prefill, PREFILL, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(batch=0)), (OK, dict(tokens=0)), (SHAPE, dict(batch=-1)), (SHAPE, dict(tokens=-1)),
    (SHAPE, dict(tokens=65)), (SHAPE, dict(heads=0)), (SHAPE, dict(prefix_len=-1)),
    (SHAPE, dict(batch=1 << 22, heads=1 << 10)), (SHAPE, dict(tokens=64, heads=1 << 20)),
    (SHAPE, dict(num_pages=-1)), (SHAPE, dict(width=-1)), (SHAPE, dict(page_tokens=0)),
    (UNSUP, dict(page_tokens=4)), (UNSUP, dict(page_tokens=48)), (UNSUP, dict(page_tokens=1 << 17)),
    (SHAPE, dict(page_stride=64 * 576 - 8)), (SHAPE, dict(page_stride=64 * 576 + 4)),
    (SHAPE, dict(num_pages=0, prefix_len=5)),
    (VALUE, dict(scale=0.0)), (VALUE, dict(scale=NAN)),
    (NULL, dict(q=None)), (NULL, dict(o=None)), (NULL, dict(kv_lens=None)), (NULL, dict(table=None)),
    (NULL, dict(cache=None)), (NULL, dict(prefix_len=5)),
    (ALIGN, dict(q=P + 8)), (ALIGN, dict(cache=P + GiB + 8)), (ALIGN, dict(o=P + 4 * GiB + 2)),
    (ALIGN, dict(kv_lens=P + 3 * GiB + 2)), (ALIGN, dict(ws=P + 5 * GiB + 8)),
    (WS, dict(ws=None)), (WS, dict(ws_bytes=1000)),
    (ALIAS, dict(o=P)), (ALIAS, dict(o=P + GiB)), (ALIAS, dict(lse=P + 4 * GiB)),
    (ALIAS, dict(ws=P + GiB)), (ALIAS, dict(o=P + 5 * GiB + 256)), (ALIAS, dict(lse=P + 3 * GiB)),
    (ALIAS, dict(prefix_table=P + 4 * GiB, prefix_len=5)),
])
def test_decode_refusals(lib, want, kw):
    assert call(lib.rda_mla_decode, DECODE, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(total=0)), (SHAPE, dict(num_seqs=0)), (SHAPE, dict(total=-1)), (SHAPE, dict(cu=None)),
    (OK, dict(cu=None, total=0)), (SHAPE, dict(kv_stride=568)), (SHAPE, dict(kv_stride=580)),
    (UNSUP, dict(page_tokens=12)), (SHAPE, dict(page_stride=100)),
    (VALUE, dict(eps=-1.0)), (VALUE, dict(eps=NAN)), (VALUE, dict(eps=INF)),
    (NULL, dict(kv=None)), (NULL, dict(kv_lens=None)), (NULL, dict(table=None)), (NULL, dict(cache=None)),
    (ALIGN, dict(kv=P + 2)), (ALIGN, dict(weight=P + 5 * GiB + 4)), (ALIGN, dict(cache=P + 4 * GiB + 8)),
    (ALIGN, dict(table=P + 3 * GiB + 1)),
    (ALIAS, dict(cache=P)), (ALIAS, dict(kv_lens=P + 4 * GiB)), (ALIAS, dict(weight=P + 4 * GiB + 64)),
    (OK, dict(num_pages=0, cache=None)), (OK, dict(width=0, table=None)),
])
def test_append_refusals(lib, want, kw):
    assert call(lib.rda_mla_append, APPEND, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(batch=0)), (SHAPE, dict(batch=-1)), (SHAPE, dict(batch=65536)), (SHAPE, dict(drafts=-1)),
    (SHAPE, dict(drafts=64)), (SHAPE, dict(vocab=0)), (SHAPE, dict(target_stride=999)),
    (SHAPE, dict(draft_stride=999)),
    (NULL, dict(target=None)), (NULL, dict(tokens=None)), (NULL, dict(uniforms=None)),
    (NULL, dict(accept=None)), (NULL, dict(out=None)),
    (WS, dict(ws=None)), (WS, dict(ws_bytes=8)),
    (ALIGN, dict(target=P + 4)), (ALIGN, dict(draft=P + GiB + 8)), (ALIGN, dict(ws=P + 6 * GiB + 8)),
    (ALIGN, dict(tokens=P + 1)), (ALIGN, dict(accept=P + 4 * GiB + 2)),
    (ALIAS, dict(accept=P)), (ALIAS, dict(out=P + GiB)), (ALIAS, dict(accept=P + 5 * GiB)),
    (ALIAS, dict(ws=P + 3 * GiB)), (ALIAS, dict(out=P + 2 * GiB)),
])
def test_verify_refusals(lib, want, kw):
    assert call(lib.rda_verify_drafts, VERIFY, **kw) == want


def test_workspace_sizes(lib):
    W = rda.rda_mla_decode_workspace_bytes
    assert W(0, 1, 32) > 0 and W(-1, 1, 32) == 0 and W(1, 65, 32) == 0 and W(1, 1, 0) == 0
    assert W(4, 1, 32, -1) == 0
    # partial sums of every query row, fp32
    assert W(256, 3, 32) >= 256 * 96 * 512 * 4
    assert W(8, 1, 32, 100) >= W(8, 1, 32) + 8 * 32 * 512 * 4
    V = rda.rda_verify_drafts_workspace_bytes
    assert V(-1, 10) == 0 and V(1, 0) == 0 and V(3, 259840) >= 3 * 64 * 16


def test_constants_match_header():
    import re
    text = open(os.path.join(os.path.dirname(rda.library_path()), "..", "include", "rda.h")).read()
    vals = {m[0]: int(m[1]) for m in re.findall(r"#define\s+(RDA_MLA_[A-Z]+(?:_[A-Z]+)?)\s+(\d+)", text)}
    assert len(vals) == 9
    for name, v in vals.items():
        assert getattr(rda, name) == v, name


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 2, 192, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rda.rda_mla_prefill(q, torch.zeros(1, 2, 256, dtype=torch.bfloat16), torch.zeros(1, 64, dtype=torch.bfloat16), 1.0)
    with pytest.raises(ValueError):
        rda.rda_mla_decode(torch.zeros(1, 1, 2, 576, dtype=torch.bfloat16), torch.zeros(1, 8, 576, dtype=torch.bfloat16),
                           torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1.0)
    with pytest.raises(ValueError):
        rda.rda_verify_drafts(torch.zeros(1, 1, 4), None, torch.zeros(1, 0, dtype=torch.int32), torch.zeros(1, 1))
    with pytest.raises(TypeError):
        rda.rda_mla_append(None, None, None, None)


def test_row_checks():
    """Rows may lie apart, their values may not."""
    x = torch.zeros(4, 3, 80)
    cpu = x.device
    assert rda._need_rows(x, "x", torch.float32, (4, 3, 80), cpu) == 240
    assert rda._need_rows(x[:, :1, 16:], "x", torch.float32, (4, 1, 64), cpu) == 240
    assert rda._need_rows(x[:1, :, :], "x", torch.float32, (1, 3, 80), cpu) == 240
    with pytest.raises(ValueError):
        rda._need_rows(x[:, :, 16:], "x", torch.float32, (4, 3, 64), cpu)
    with pytest.raises(ValueError):
        rda._need_rows(x.transpose(1, 2), "x", torch.float32, (4, 80, 3), cpu)
    with pytest.raises(ValueError):
        rda._need_rows(x, "x", torch.float32, (4, 3, 81), cpu)
    with pytest.raises(TypeError):
        rda._need_rows(x, "x", torch.bfloat16, (4, 3, 80), cpu)
    p = torch.zeros(2, 3, 10)
    assert rda._prob_rows(p, "p", (2, 3, 10), cpu) == 10
    assert rda._prob_rows(p[..., :7], "p", (2, 3, 7), cpu) == 10
    assert rda._prob_rows(p[:, :1], "p", (2, 1, 10), cpu) == 30
    with pytest.raises(ValueError):
        rda._prob_rows(p[:, :2], "p", (2, 2, 10), cpu)
    with pytest.raises(TypeError):
        rda._prob_rows(p.double(), "p", (2, 3, 10), cpu)


def test_decode_plan_divides_all_work(lib):
    """ctypes smoke: sizes near the limits do not overflow the plan."""
    size = lib.rda_mla_decode_workspace_bytes
    assert size.restype is ctypes.c_size_t
    assert rda.rda_mla_decode_workspace_bytes(1 << 14, 64, 64) > (1 << 26) * 512 * 4
