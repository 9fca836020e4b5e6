"""GPU tests of rda_mla_decode over caches of hundreds of thousands of rows,
one sequence's own and shared ones.  The queries are spread so that a few rows
hold most of the weight: the outputs are then far larger than the bound, which
grows with the number of rows."""
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


def run(dev, lens, T, H, page, prefix, seed):
    say(f"[mla decode] long: lens={lens} T={T} H={H} page={page} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, page, seed, prefix, spread=4.0)
    # query 0 of the last token and head finds the last row that it sees
    last = lens[0] - 1
    cache[int(table[0, last // page]), last % page] = 0.25 * q[0, T - 1, H - 1]
    o, lse = rda.rda_mla_decode(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=prefix,
                                want_lse=True)
    torch.cuda.synchronize()
    ro, rl, bo, bl = mla_ref.decode(q.cpu(), cache.cpu(), table.cpu(), lens, SCALE,
                                    None if pre is None else pre.cpu(), prefix)
    assert float(ro.abs().amax(-1).min()) > 8 * float(bo.amax()), "the bound says something"
    mla_ref.check("o", o, ro, bo)
    mla_ref.check("lse", lse, rl, bl)


@pytest.mark.parametrize("lens,T,H,page,prefix", [
    ([262144], 1, 2, 64, 0),
    ([200003, 7, 4099], 1, 2, 256, 0),
    ([131075], 2, 2, 16, 0),
    ([90, 1], 1, 2, 64, 262001),
])
def test_long(dev, lens, T, H, page, prefix):
    run(dev, lens, T, H, page, prefix, 20 + T + page)
