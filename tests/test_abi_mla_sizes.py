"""Calls of the latent-attention entry points that would need more workgroups
than one launch holds are refused before anything reaches a device (CPU)."""
import pytest

from test_abi_mla import APPEND, PREFILL, OK, SHAPE, call, lib  # noqa: F401


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(num_seqs=1 << 24, heads=1, q_stride=192, kv_stride=256)),
    (SHAPE, dict(num_seqs=(1 << 31) - 1, heads=1, q_stride=192, kv_stride=256)),
    (SHAPE, dict(num_seqs=1 << 20, heads=16, q_stride=16 * 192, kv_stride=16 * 256)),
    (OK, dict(num_seqs=(1 << 20) - 1, heads=16, q_stride=16 * 192, kv_stride=16 * 256)),
    (SHAPE, dict(num_seqs=1, heads=8, q_stride=8 * 192, kv_stride=8 * 256, total_q=1 << 28)),
])
def test_prefill(lib, want, kw):  # noqa: F811
    assert call(lib.rda_mla_prefill, PREFILL, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(total=(1 << 25) + 1)), (SHAPE, dict(total=(1 << 31) - 1)),
    (OK, dict(total=0, num_seqs=(1 << 31) - 1)),
])
def test_append(lib, want, kw):  # noqa: F811
    assert call(lib.rda_mla_append, APPEND, **kw) == want
