"""GPU tests of rda_mla_prefill's kernels where queries or keys that are seen
hold NaN, and over keys of one sequence in the hundreds of thousands."""
import pytest
import torch

import mla_ref
from gated_delta_amd import rda
from gpu_util import need_gpu, say
from test_gpu_mla_prefill_wide import SCALE, compare, make, offsets

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.mark.parametrize("lq,lk,H", [
    ([70, 3], [200, 3], 4),         # a workgroup to a CU
    ([400, 300], [400, 500], 80),   # two to a CU
    ([2300], [2300], 64),           # 256 queries a workgroup
])
def test_nan_query(dev, lq, lk, H):
    """The query that holds NaN gets NaN; those of its block keep their values."""
    say(f"[mla prefill] NaN query lq={lq} lk={lk} H={H}")
    q, kv, pe = make(dev, lq, lk, H, 1)
    hit = [0, 37, lq[0] - 1]
    q[hit[0], 1, 191], q[hit[1], 1, 0], q[hit[2], 1, 64] = NAN, NAN, NAN
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, offsets(lq), offsets(lk), want_lse=True)
    torch.cuda.synchronize()
    rows = sorted({0, 1, 36, 37, 38, 63, 64, lq[0] - 2, lq[0] - 1} & set(range(lq[0])))
    compare(o[:lq[0]], lse[:lq[0]], q[:lq[0]], kv[:lk[0]], pe[:lk[0]], lq[:1], lk[:1], True, (0, 1, 2), rows=rows)
    assert bool(torch.isnan(o[hit, 1]).all()) and bool(torch.isnan(lse[hit, 1]).all())


@pytest.mark.parametrize("lq,lk,H", [([70], [70], 4), ([700], [700], 80), ([2300], [2300], 64)])
def test_nan_key(dev, lq, lk, H):
    """Every query that sees a key with NaN gets NaN, output and log-sum-exp."""
    say(f"[mla prefill] NaN key lq={lq} H={H}")
    q, kv, pe = make(dev, lq, lk, H, 2)
    at = lq[0] - 20
    kv[at, 1, 3] = NAN
    pe[5, 1] = NAN
    kv[at, 2, 127] = NAN
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, want_lse=True)
    torch.cuda.synchronize()
    assert bool(torch.isnan(o[5:]).all()) and bool(torch.isnan(lse[5:]).all())
    assert bool(torch.isfinite(o[:5].float()).all()) and bool(torch.isfinite(lse[:5]).all())
    pe[5, 1] = 0
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, want_lse=True)
    torch.cuda.synchronize()
    for h in (1, 2):
        assert bool(torch.isnan(o[at:, h]).all()) and bool(torch.isnan(lse[at:, h]).all())
    rows = [0, 4, at - 1, at, lq[0] - 1]
    compare(o, lse, q, kv, pe, lq, lk, True, (0, 1), rows=rows)


@pytest.mark.parametrize("lq,lk", [([3], [262147]), ([1, 130], [200001, 70000])])
def test_long(dev, lq, lk):
    say(f"[mla prefill] long lq={lq} lk={lk}")
    q, kv, pe = make(dev, lq, lk, 2, 3, spread=5.0)
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, offsets(lq), offsets(lk), want_lse=True)
    torch.cuda.synchronize()
    q, kv, pe = q.cpu(), kv.cpu(), pe.cpu()
    for a, c, n, m in zip(offsets(lq), offsets(lk), lq, lk):
        at = sorted({0, n // 2, n - 1})
        k = torch.cat([kv[c:c + m, 1, :128], pe[c:c + m]], 1)
        ro, rl, bo, bl = mla_ref.attend(q[a:a + n, 1][at], k, kv[c:c + m, 1, 128:], SCALE, [i + 1 + m - n for i in at])
        assert bool((ro.abs().amax(-1) > 8 * bo.amax(-1)).all())   # each row, so its bound says something
        mla_ref.check("o", o[a:a + n, 1].cpu()[at], ro, bo)
        mla_ref.check("lse", lse[a:a + n, 1].cpu()[at], rl, bl)
