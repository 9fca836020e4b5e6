"""GPU tests of rda_mla_decode_q4 at the smallest scales: every positive finite
scale weighs the rows that are seen, one whose products with the scores all but
vanish alike (the mean of the rows, and the logarithm of their number)."""
import pytest
import torch

import mla_q4_ref as ref
from gated_delta_amd import rda
from gpu_util import need_gpu, say
from test_gpu_mla_decode_q4 import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.mark.parametrize("scale", [1.8e-38, 1.2e-38, 1e-42, 1.5e-45])
@pytest.mark.parametrize("lens,T,H,prefix", [
    ([20, 33, 0], 1, 5, 0),        # a piece a sequence: outputs at once
    ([1, 2, 40], 3, 40, 0),        # 64 query rows a workgroup
    ([777], 1, 8, 0),              # many pieces, joined by 16 waves
    ([1500, 40], 1, 100, 0),       # by four
    ([700] * 20, 1, 32, 0),        # by one
    ([20, 0, 70], 1, 8, 300),      # behind a prefix
    ([20, 0, 70], 2, 40, 300),
])
def test_least_scales(dev, scale, lens, T, H, prefix):
    say(f"[mla q4] scale={scale} lens={lens[:4]} T={T} H={H} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, 16, 31, prefix)
    o, lse = rda.rda_mla_decode_q4(q, cache, table, kl, scale, prefix_table=pre, prefix_len=prefix, want_lse=True)
    ro, rl, bo, bl = ref.decode(q, cache, table.cpu(), lens, scale, None if pre is None else pre.cpu(), prefix)
    ref.check("o", o, ro, bo)
    ref.check("lse", lse, rl, bl)
