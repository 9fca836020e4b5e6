"""GPU tests of rda_mla_decode where rows or queries that are seen hold
infinities or NaN: the result is the formula's, however the sequence's tiles
are shared out over workgroups and joined."""
import pytest
import torch

import mla_ref
from gated_delta_amd import rda
from gpu_util import need_gpu, say
from test_gpu_mla_decode import SCALE, make

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def put(cache, table, row, channel, value):
    page = cache.shape[1]
    cache[int(table[row // page]), row % page, channel] = value


def compare(q, cache, table, kl, pre, prefix):
    lens = kl.tolist()
    o, lse = rda.rda_mla_decode(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=prefix,
                                want_lse=True)
    torch.cuda.synchronize()
    ro, rl, bo, bl = mla_ref.decode(q.cpu(), cache.cpu(), table.cpu(), lens, SCALE,
                                    None if pre is None else pre.cpu(), prefix)
    mla_ref.check("o", o, ro, bo)
    mla_ref.check("lse", lse, rl, bl)
    return o, lse


@pytest.mark.parametrize("lens,T,H,prefix", [
    ([20], 1, 4, 0), ([257], 1, 4, 0), ([777], 1, 32, 0), ([777, 5, 0], 1, 40, 0), ([300, 40], 3, 16, 0),
    ([900, 257], 2, 64, 0), ([9, 0], 1, 4, 300), ([257, 30], 2, 40, 65),
])
def test_nan_query(dev, lens, T, H, prefix):
    """A query that holds NaN gets NaN where it sees any key, and the queries
    beside it keep their values."""
    say(f"[mla decode] NaN query lens={lens} T={T} H={H} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, 16, sum(lens), prefix)
    q[:, T - 1, 1, 3] = NAN
    q[0, 0, 0, 575] = NAN
    o, lse = compare(q, cache, table, kl, pre, prefix)
    assert bool(torch.isnan(o[0, 0, 0]).all()) and bool(torch.isnan(lse[0, 0, 0]))


@pytest.mark.parametrize("channel", [0, 511, 512])
@pytest.mark.parametrize("lens,T,H,prefix,row", [
    ([257], 1, 4, 0, 256),        # the only visible row of the last share
    ([257], 1, 4, 0, 0),
    ([777], 1, 32, 0, 776),
    ([777], 1, 32, 0, 400),
    ([20], 1, 4, 0, 19),
    ([33], 1, 8, 40, 32),
    ([300], 2, 80, 0, 298),       # seen by both new tokens
    ([300], 3, 16, 0, 298),       # by all but the first
    ([257], 2, 16, 0, 256),       # by the last
])
def test_nan_row(dev, lens, T, H, prefix, row, channel):
    say(f"[mla decode] NaN in row {row} channel {channel} lens={lens} T={T} H={H} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, 16, 7, prefix)
    put(cache, table[0], row, channel, NAN)
    o, lse = compare(q, cache, table, kl, pre, prefix)
    assert bool(torch.isnan(o[0, T - 1]).all()) and bool(torch.isnan(lse[0, T - 1]).all())


@pytest.mark.parametrize("prefix,row", [(1, 0), (300, 299), (700, 31)])
def test_nan_prefix_row(dev, prefix, row):
    q, cache, table, kl, pre = make(dev, [40, 0, 3], 1, 32, 16, 8, prefix)
    put(cache, pre, row, 512, NAN)
    o, lse = compare(q, cache, table, kl, pre, prefix)
    assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("n,bad", [(257, 256), (20, 19), (777, 400)])
def test_row_of_score_minus_infinity(dev, n, bad):
    """An infinity that meets a query channel of the other sign: the score is
    -inf and its probability 0, so only 0 * inf in that channel shows it."""
    say(f"[mla decode] score -inf at row {bad} of {n}")
    H = 4
    q, cache, table, kl, _ = make(dev, [n], 1, H, 16, 9)
    q[..., 5] = -q[..., 5].abs() - 1
    put(cache, table[0], bad, 5, INF)
    o, lse = rda.rda_mla_decode(q, cache, table, kl, SCALE, want_lse=True)
    torch.cuda.synchronize()
    rows = mla_ref.cached_rows(cache.cpu(), table[0].cpu(), n)
    rows = torch.cat([rows[:bad], rows[bad + 1:]])
    ro, rl, bo, bl = mla_ref.attend(q[0, 0], rows, rows[:, :512], SCALE, [n - 1] * H)
    ro[:, 5] = NAN
    mla_ref.check("o", o[0, 0], ro, bo)
    mla_ref.check("lse", lse[0, 0], rl, bl)
