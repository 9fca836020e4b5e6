"""GPU tests of rda_mla_append_q4 with norm weights that are not finite, against
the 64-bit form byte for byte: 32 channels among which the normed values hold an
infinity or NaN become NaN, whatever the row's own values are."""
import math

import pytest
import torch

from gpu_util import need_gpu, say
from test_gpu_mla_q4 import append, norm_weight, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("channels", [[0], [37], [511], [5, 100, 101, 300], list(range(512))])
def test_bad_weight(dev, bad, channels):
    say(f"[append q4] weight {bad} at {channels[:4]}")
    weight = norm_weight(20)
    weight[channels] = bad
    got, table, _, _ = append(dev, rows(40, 21), [40], [40], 16, weight)
    hit = sorted({c // 32 for c in channels})
    scales = got[table[0].long().to(dev)].reshape(-1, 400)[:40, 256:272]
    assert bool((scales[:, hit] == 255).all()) and int((scales == 255).sum()) == 40 * len(hit)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_bad_weight_on_zero(dev, bad):
    """Zero times an infinity is NaN; a group of zeros stays one under a finite weight."""
    say(f"[append q4] weight {bad} on zeros")
    kv, weight = rows(24, 22), norm_weight(23)
    kv[:, 64] = 0.0
    kv[::2, 130] = -0.0
    kv[::3, 256:288] = 0.0
    weight[[64, 130, 270]] = bad
    append(dev, kv, [24], [24], 8, weight)


@pytest.mark.parametrize("weight,eps", [(2.0 ** 124, 1e-5), (2.0 ** 126, 0.0), (3.4e38, 1e-5)])
def test_largest_values(dev, weight, eps):
    """Values beyond 7 x 2^125 become 6 x 2^125; no finite value becomes NaN."""
    say(f"[append q4] weights of {weight}")
    kv = rows(20, 24)
    kv[::4, 70] = 30.0                     # beside small ones
    kv[5:9] *= 1e-30
    w = torch.full((512,), weight) * torch.where(torch.arange(512) % 3 == 0, -1.0, 1.0)
    got, table, _, _ = append(dev, kv, [20], [20], 8, w, eps=eps)
    assert int(got[table[0].long().to(dev)].reshape(-1, 400)[:20, 256:272].max()) == 125 + 127
    append(dev, torch.full((3, 576), 3.3895e38).bfloat16(), [3], [3], 8, None)
