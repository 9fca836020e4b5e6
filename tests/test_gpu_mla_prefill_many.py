"""GPU tests of rda_mla_prefill at batches with more query blocks than CUs but
sequences too short for the blocks of 256 queries: two workgroups share a CU."""
import pytest
import torch

from gated_delta_amd import rda
from gpu_util import need_gpu, say
from test_gpu_mla_prefill_wide import SCALE, compare, make, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.mark.parametrize("lq,lk,H", [
    ([300, 1, 65], [300, 1, 65], 64),
    ([129, 0, 70, 128], [400, 50, 70, 131], 64),
    ([1] * 40, [1, 2, 63, 64, 65, 127, 128, 129, 0, 193] * 4, 16),
    ([10, 200, 33], [4, 260, 0], 80),                       # rows that see nothing
    ([1100], [1100], 40),
])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_and_heads(dev, lq, lk, H, causal):
    say(f"[mla prefill many] lq={lq} lk={lk} H={H} causal={causal}")
    q, kv, pe = make(dev, lq, lk, H, sum(lq) + H)
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, offsets(lq), offsets(lk), causal=causal, want_lse=True)
    torch.cuda.synchronize()
    compare(o, lse, q, kv, pe, lq, lk, causal, (0, H - 1))


@pytest.mark.parametrize("spread", [0.0, 60.0])
def test_large_scores(dev, spread):
    q, kv, pe = make(dev, [500], [500], 80, 3, spread)
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, want_lse=True)
    compare(o, lse, q, kv, pe, [500], [500], True, (0, 79))


def test_growing_scores(dev):
    T, H = 600, 64
    q, kv, pe = make(dev, [T], [T], H, 5)
    q, pe = q * 0 + 1, pe * 0
    kv[:, :, :128] = (torch.arange(T, device=dev).float() * 0.01).bfloat16()[:, None, None]
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE * 20, want_lse=True)
    compare(o, lse, q, kv, pe, [T], [T], True, (0,), scale=SCALE * 20)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_bad_values_in_masked_places(dev, bad):
    T, H = 500, 80
    for at in (63, 64, 130, 499):
        q, kv, pe = make(dev, [T], [T], H, 6)
        clean, _ = rda.rda_mla_prefill(q, kv, pe, SCALE)
        kv[at, 1] = bad
        kv[at, 2, 128 + 7] = bad
        o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, want_lse=True)
        for h in (1, 2):
            assert bool(torch.isfinite(o[:at, h].float()).all()), (at, h)
        near = [i for i in (0, at - 40, at - 1) if 0 <= i < at]
        compare(o, lse, q, kv, pe, [T], [T], True, (1, 2), rows=near)
        assert torch.equal(o[:, 0], clean[:, 0]) and torch.equal(o[:, 3:], clean[:, 3:])
        assert not bool(torch.isfinite(o[at:, 2, 7].float()).any())
        assert bool(torch.isfinite(o[at:, 2, 8:].float()).all())
