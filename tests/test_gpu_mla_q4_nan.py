"""GPU tests of rda_mla_decode_q4 where queries or cached rows hold infinities
or NaN: the formula's result where they are seen, and no trace where they are
not, however the tiles are shared out and joined."""
import pytest
import torch

import mla_q4_ref as ref
from gated_delta_amd import rda
from gpu_util import need_gpu, say
from test_gpu_mla_decode_q4 import SCALE, make

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def put_group(cache, table, row, group):
    """A group of 32 channels as the writer leaves it for an infinity or NaN."""
    page = cache.shape[1]
    at = cache[int(table[row // page]), row % page]
    at[16 * group:16 * group + 16] = 0
    at[256 + group] = 255


def put_pe(cache, table, row, channel, value):
    page = cache.shape[1]
    at = 272 + 2 * channel
    cache[int(table[row // page]), row % page, at:at + 2] = \
        torch.tensor([value], dtype=torch.bfloat16).view(torch.uint8).to(cache.device)


def decode(q, cache, table, kl, pre, prefix):
    o, lse = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=prefix, want_lse=True)
    torch.cuda.synchronize()
    return o, lse


def expect(q, cache, table, kl, pre, prefix):
    return ref.decode(q, cache, table.cpu(), kl.tolist(), SCALE, None if pre is None else pre.cpu(), prefix)


def compare(*args):
    o, lse = decode(*args)
    ro, rl, bo, bl = expect(*args)
    ref.check("o", o, ro, bo)
    ref.check("lse", lse, rl, bl)
    return o, lse


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("lens,T,H,prefix", [
    ([20], 1, 4, 0), ([257], 1, 4, 0), ([777], 1, 32, 0), ([777, 5, 0], 1, 40, 0), ([300, 40], 3, 32, 0),
    ([9, 0], 1, 4, 300), ([257, 30], 2, 40, 65),
])
def test_query(dev, lens, T, H, prefix, bad):
    """A query whose latent part holds NaN or an infinity gets NaN where it sees any
    key, and the queries beside it keep their values."""
    say(f"[mla q4] query {bad} lens={lens} T={T} H={H} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, 16, sum(lens), prefix)
    want = expect(q, cache, table, kl, pre, prefix)
    hit = torch.zeros(len(lens), T, H, dtype=torch.bool)
    hit[:, T - 1, 1] = hit[0, 0, 0] = True
    q[:, T - 1, 1, 3] = bad
    q[0, 0, 0, 511] = bad
    o, lse = (x.cpu() for x in decode(q, cache, table, kl, pre, prefix))
    none = torch.isinf(want[1])   # no key
    for x, w, b, name in ((o, want[0], want[2], "o"), (lse, want[1], want[3], "lse")):
        ref.check(name, x[~hit | none], w[~hit | none], b[~hit | none])
        assert bool(torch.isnan(x[hit & ~none].float()).all())


def test_query_shared_channel(dev):
    q, cache, table, kl, _ = make(dev, [300, 20], 1, 5, 16, 3)
    want = expect(q, cache, table, kl, None, 0)
    q[0, 0, 2, 575] = NAN
    o, lse = (x.cpu() for x in decode(q, cache, table, kl, None, 0))
    assert bool(torch.isnan(o[0, 0, 2].float()).all()) and bool(torch.isnan(lse[0, 0, 2]))
    keep = [0, 1, 3, 4]
    ref.check("o", o[:, :, keep], want[0][:, :, keep], want[2][:, :, keep])


@pytest.mark.parametrize("where", [0, 5, 15, "pe"])
@pytest.mark.parametrize("lens,T,H,prefix,row", [
    ([257], 1, 4, 0, 256),        # the only visible row of the last tile
    ([257], 1, 4, 0, 0),
    ([777], 1, 32, 0, 776),
    ([777], 1, 32, 0, 400),
    ([20], 1, 4, 0, 19),
    ([33], 1, 8, 40, 32),
    ([300], 2, 80, 0, 298),       # seen by both new tokens
    ([300], 3, 16, 0, 298),       # by all but the first
    ([257], 2, 16, 0, 256),       # by the last
    ([500, 70], 1, 64, 0, 301),
])
def test_row(dev, lens, T, H, prefix, row, where):
    say(f"[mla q4] NaN in row {row} at {where} lens={lens} T={T} H={H} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, 16, 7, prefix)
    clean = decode(q, cache, table, kl, pre, prefix)
    if where == "pe":
        put_pe(cache, table[0], row, 0, NAN)
    else:
        put_group(cache, table[0], row, where)
    o, lse = compare(q, cache, table, kl, pre, prefix)
    sees = [lens[0] - (T - 1 - t) > row for t in range(T)]
    for t in range(T):
        if sees[t]:
            assert bool(torch.isnan(o[0, t]).all()) and bool(torch.isnan(lse[0, t]).all())
        else:       # bit for bit as without it
            assert torch.equal(o[0, t], clean[0][0, t]) and torch.equal(lse[0, t], clean[1][0, t])
    assert torch.equal(o[1:], clean[0][1:])


@pytest.mark.parametrize("prefix,row", [(1, 0), (300, 299), (700, 31)])
@pytest.mark.parametrize("H", [32, 72])
def test_prefix_row(dev, prefix, row, H):
    q, cache, table, kl, pre = make(dev, [40, 0, 3], 1, H, 16, 8, prefix)
    put_group(cache, pre, row, 7)
    o, lse = compare(q, cache, table, kl, pre, prefix)
    assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("n,bad", [(257, 256), (20, 19), (777, 400), (33, 0)])
def test_row_of_score_minus_infinity(dev, n, bad):
    """An infinity among the shared channels that meets a query channel of the other
    sign: the row weighs nothing, and as the shared channels are no values, the
    result is that without it."""
    say(f"[mla q4] score -inf at row {bad} of {n}")
    H = 4
    q, cache, table, kl, _ = make(dev, [n], 1, H, 16, 9)
    q[..., 517] = -q[..., 517].abs() - 1
    put_pe(cache, table[0], bad, 5, INF)
    o, lse = decode(q, cache, table, kl, None, 0)
    rows = ref.cached(cache.cpu(), table[0].cpu(), n)
    rows = torch.cat([rows[:bad], rows[bad + 1:]])
    ro, rl, bo, bl = ref.attend(q[0, 0], rows, rows[:, :512], SCALE)
    ref.check("o", o[0, 0], ro, bo)
    ref.check("lse", lse[0, 0], rl, bl)


@pytest.mark.parametrize("B,low,high,T,H", [(300, 2, 120, 2, 4), (250, 40, 300, 3, 4), (130, 30, 400, 2, 40)])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_masked_places_of_many(dev, B, low, high, T, H, bad):
    """The last row, which the last token alone sees, where workgroups take pieces of
    several sequences."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(low, high + 1, (B,), generator=g).tolist()
    say(f"[mla q4] masked places B={B} T={T} H={H} bad={bad}")
    q, cache, table, kl, _ = make(dev, lens, T, H, 16, B)
    clean = decode(q, cache, table, kl, None, 0)
    hit = list(range(0, B, 7))
    for b in hit:
        (put_group(cache, table[b], lens[b] - 1, 3) if bad is NAN else put_pe(cache, table[b], lens[b] - 1, 9, bad))
    o, lse = decode(q, cache, table, kl, None, 0)
    same = torch.ones(B, T, dtype=torch.bool, device=dev)
    same[hit, T - 1] = False
    assert torch.equal(o[same], clean[0][same]) and torch.equal(lse[same], clean[1][same])
    if bad is NAN:
        assert bool(torch.isnan(o[~same]).all()) and bool(torch.isnan(lse[~same]).all())
