"""GPU tests of the 4-bit cache's reader and attention on two streams at once, in
turn without a wait, and of the attention's plan by workgroups of 64 query
rows for more sequences than such a workgroup has threads."""
import pytest
import torch

from gated_delta_amd import rda
from gpu_util import need_gpu, say
from test_gpu_mla_decode_q4 import SCALE, make, run
from test_gpu_mla_q4_shares import spread
from test_gpu_mla_streams import alternate, equal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.mark.parametrize("prefix", [0, 500])
@pytest.mark.parametrize("H", [32, 40])
def test_read_and_decode(dev, prefix, H):
    """Two batches of other lengths, so that a workspace shared by mistake would hold
    other plans; what the reader gives is compared too."""
    say(f"[mla q4 streams] read and decode, prefix={prefix} H={H}")
    args = [make(dev, lens, 1, H, 64, 3, prefix) for lens in ([700, 300, 2000], [1500, 1, 40])]

    def fn(s, which):
        q, cache, table, kl, pre = args[which]
        rows = rda.rda_mla_read_q4(cache, table, kl, 50 + which, [0, 40, 49, 50 + which], stream=s)
        o, lse = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=prefix, want_lse=True,
                                       stream=s)
        return rows.view(torch.int16), o, lse

    want = fn(None, 0) + fn(None, 1)
    torch.cuda.synchronize()
    assert not bool(torch.isnan(want[1]).any()) and not bool(torch.isnan(want[4]).any())
    alternate(lambda s: fn(s, 0) + fn(s, 1), want, equal)


@pytest.mark.parametrize("n,T,H,prefix", [(600, 1, 40, 0), (1030, 1, 33, 0), (513, 2, 20, 70), (600, 3, 24, 0)])
def test_many_sequences(dev, n, T, H, prefix):
    run(dev, spread(n, 0, 90, n), T, H, 32, seed=n, prefix=prefix)
