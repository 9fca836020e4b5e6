"""GPU tests of rda_mla_decode where workgroups take pieces of several
sequences: infinities and NaN in the rows that only the last new token sees, and
the same results whatever else is in the batch's workspace."""
import pytest
import torch

import mla_ref
from gated_delta_amd import rda
from gpu_util import need_gpu, say
from test_gpu_mla_decode import SCALE, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.mark.parametrize("B,low,high,T,H", [(300, 2, 120, 2, 4), (250, 40, 300, 3, 4), (130, 30, 400, 2, 40)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_in_masked_places(dev, B, low, high, T, H, bad):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(low, high + 1, (B,), generator=g).tolist()
    say(f"[mla decode shares] B={B} T={T} H={H} bad={bad}")
    q, cache, table, kl, _ = make(dev, lens, T, H, 16, B)
    hit = list(range(0, B, 7))
    for b in hit:      # the last row, which the last token alone sees
        n = lens[b] - 1
        cache[int(table[b, n // 16]), n % 16, 5] = bad
    ws = torch.full((rda.rda_mla_decode_workspace_bytes(B, T, H, 0),), 255, dtype=torch.uint8, device=dev)
    o, lse = rda.rda_mla_decode(q, cache, table, kl, SCALE, want_lse=True, workspace=ws)
    again, _ = rda.rda_mla_decode(q, cache, table, kl, SCALE, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(o[:, :T - 1], again[:, :T - 1])
    clean = torch.ones(B, T, dtype=torch.bool)
    clean[hit, T - 1] = False
    ro, rl, bo, bl = mla_ref.decode(q.cpu(), cache.cpu(), table.cpu(), lens, SCALE)
    mla_ref.check("o", o.cpu()[clean], ro[clean], bo[clean])
    mla_ref.check("lse", lse.cpu()[clean], rl[clean], bl[clean])
    assert not torch.isfinite(o.cpu()[hit, T - 1][..., 5].float()).any()
