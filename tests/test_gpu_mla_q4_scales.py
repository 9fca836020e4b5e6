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


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 20, 2.0 ** 24])
@pytest.mark.parametrize("lens,prefix", [([1] * 9, 0), ([1] * 70, 0), ([0] * 9, 1)])
def test_large_scores(dev, size, lens, prefix):
    """One row each, with scores up to 2^28 of either sign: log-sum-exp is the score.
    The score's products in 24 bits (200 sums), c = scale log2 e, s c, ln 2 and the last
    product, 2^-24 each (a sum's cut 2^-23); the sum of the probabilities is
    2^(what s c was rounded by), in its logarithm once more 2^-22."""
    say(f"[mla q4] scores of {size} and more")
    q, cache, table, kl, pre = make(dev, lens, 1, 7, 16, 33, prefix)
    cache[..., 256:272] = torch.where(cache[..., 256:272] == 255, 255, 127).to(torch.uint8)
    q.copy_((q.float() * size).bfloat16())
    o, lse = rda.rda_mla_decode_q4(q, cache, table, kl, 0.25, prefix_table=pre, prefix_len=prefix, want_lse=True)
    rows = [ref.cached(cache.cpu(), (table[b] if n else pre).cpu(), 1)[0] for b, n in enumerate(lens)]
    keys = torch.stack(rows)[:, None, None]
    y = q.cpu().double()
    want, most = 0.25 * (y * keys).sum(-1), 0.25 * (y * keys).abs().sum(-1)
    assert float(want.abs().max()) < 2.0 ** 28
    lost = 0.25 * 512 * 4 * 2.0 ** -14 * y[..., :512].abs().amax(-1)   # small channels: |v| / 2 + u is 4 at most
    err = (lse.cpu().double() - want).abs()
    assert bool((err <= 200 * 2.0 ** -23 * most + lost + 8 * 2.0 ** -24 * want.abs() + 2.0 ** -22).all())
    v = keys[..., :512].expand(o.shape)
    assert bool(((o.cpu().double() - v).abs() <= 2.0 ** -7 * v.abs()).all())
