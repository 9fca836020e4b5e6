"""GPU tests of rda_mla_append_q4 and rda_mla_read_q4 (the 4-bit latent cache's
writer and reader) against the 64-bit forms, byte for byte: a code is a choice
between neighbours far apart, and the kernel makes it in 64 bits too."""
import math

import pytest
import torch

import mla_q4_ref as ref
from gated_delta_amd import rda
from gpu_util import guarded, need_gpu, say

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def offsets(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


def tables(after, page, seed, spare=2):
    """A block table over shuffled pages, the pages of the pool."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in after]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g).tolist()
    table = torch.full((len(after), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for n, k in enumerate(need):
        table[n, :k] = torch.tensor(perm[at:at + k], dtype=torch.int32)
        at += k
    return table, pool


def append(dev, kv, new, after, page, weight, seed=0, equal=False, eps=EPS, stride=None):
    """One call into a pool of 0xa5 bytes; every byte of the pool is compared."""
    table, pool = tables(after, page, seed)
    cache = guarded((pool, page, 400), torch.uint8, dev)
    cache.t.fill_(0xA5)
    lens = torch.tensor(after, dtype=torch.int32, device=dev)
    cu = None if equal else torch.tensor(offsets(new), dtype=torch.int32, device=dev)
    want = ref.append(kv, cache.t, table, after, offsets(new), weight, eps)
    x = kv.to(dev)
    if stride:
        wide = torch.full((kv.shape[0], stride), float("nan"), dtype=torch.bfloat16, device=dev)
        wide[:, 8:584] = x
        x = wide[:, 8:584]
    got = rda.rda_mla_append_q4(x, cache.t, table.to(dev), lens, cu,
                                weight=None if weight is None else weight.to(dev), eps=eps)
    torch.cuda.synchronize()
    assert got is cache.t
    cache.check("cache")
    assert torch.equal(got.cpu(), want)
    return got, table, lens, cu


def rows(n, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(n, 576, generator=g)).bfloat16()


def norm_weight(seed):
    return 1 + 0.2 * torch.randn(512, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("new,after,page,equal", [
    ([1], [1], 8, True), ([1], [65], 64, True), ([3, 3], [3, 70], 16, True), ([1] * 9, list(range(1, 10)), 8, True),
    ([5, 0, 130, 1], [5, 20, 200, 64], 64, False), ([0, 0, 7], [0, 3, 7], 256, False),
    ([1, 2] * 70, [9, 40] * 70, 16, False)])
@pytest.mark.parametrize("normed", [True, False])
def test_append(dev, new, after, page, equal, normed):
    say(f"[append q4] new={new[:8]} after={after[:8]} page={page} normed={normed}")
    append(dev, rows(sum(new), len(new)), new, after, page, norm_weight(1) if normed else None, equal=equal)


@pytest.mark.parametrize("spread", [1e-30, 1e-3, 1.0, 1e4, 1e30])
def test_magnitudes(dev, spread):
    say(f"[append q4] spread={spread}")
    append(dev, rows(20, 5, spread), [20], [20], 32, None)
    append(dev, rows(20, 6, spread), [20], [20], 32, norm_weight(2))
    append(dev, rows(20, 6, spread), [20], [20], 32, norm_weight(2), eps=0.0)


def test_borders(dev):
    """Every bf16 mantissa against every scale position: half-way values, the largest
    of a group just below, at and above 7 / 4 of a power of two."""
    say("[append q4] borders")
    kv = torch.zeros(256, 576)
    for i in range(128):
        top = (128 + i) / 128
        for g in range(16):
            kv[i, 32 * g] = top * 2.0 ** (g - 8)
            kv[i, 32 * g + 1:32 * g + 32] = torch.tensor(
                [x * 2.0 ** (g - 8) * s for x in (1 / 16, 3 / 16, 5 / 16, 7 / 16, 5 / 8, 7 / 8, 5 / 4, 1 / 8, 3 / 8,
                                                  15 / 16, 17 / 16, 1 / 32, 3 / 32, 3 / 4, 1.0) for s in (1, -1)] + [0.0])
        kv[128 + i, :512] = -kv[i, :512].flip(0)
    append(dev, kv.bfloat16(), [256], [256], 64, None)


def test_extremes(dev):
    """Zeros (of both signs), the least and largest bf16, infinities and NaN."""
    say("[append q4] extremes")
    kv = rows(12, 9)
    kv[0, :512] = 0.0
    kv[1, :512] = -0.0
    kv[2, :512] = 1e-40                    # subnormal
    kv[3, :512] = 3.3895e38
    kv[4, 5] = math.inf
    kv[5, 40] = -math.inf
    kv[6, 100] = math.nan
    kv[7, 511] = 3.3895e38
    kv[8, 520] = math.nan                  # a shared channel is copied
    kv[9, 32:64] = 0.0
    kv[10, :512] = 1e-36
    append(dev, kv, [12], [12], 16, None)
    kv[4:7] = rows(3, 10)
    append(dev, kv, [12], [12], 16, norm_weight(3))


def test_norm_of_bad_rows(dev):
    """An infinity or NaN reaches the norm: every group of the row is NaN."""
    say("[append q4] norm of bad rows")
    kv = rows(2, 11)
    kv[0, 3], kv[1, 300] = math.inf, math.nan
    cache = torch.zeros(1, 8, 400, dtype=torch.uint8, device=dev)
    table = torch.zeros(1, 1, dtype=torch.int32, device=dev)
    lens = torch.tensor([2], dtype=torch.int32, device=dev)
    rda.rda_mla_append_q4(kv.to(dev), cache, table, lens, weight=norm_weight(4).to(dev))
    out = rda.rda_mla_read_q4(cache, table, lens, 2)
    # the row with an infinity: x / inf is 0, inf / inf is NaN
    assert bool(torch.isnan(out[1, :512]).all())
    assert bool(torch.isnan(out[0, :32]).all()) and float(out[0, 32:512].float().abs().max()) == 0


def test_strided_rows(dev):
    say("[append q4] strided rows")
    append(dev, rows(40, 12), [40], [47], 16, norm_weight(5), stride=640)


def test_out_of_range(dev):
    """Positions and page ids out of range are not written."""
    say("[append q4] out of range")
    kv, page = rows(30, 13), 8
    cache = torch.full((3, page, 400), 0xA5, dtype=torch.uint8, device=dev)
    table = torch.tensor([[0, -1], [7, 2], [1, 1]], dtype=torch.int32)
    after, cu = [12, 16, 20], [0, 10, 20, 30]
    want = ref.append(kv, cache, table, after, cu, None, EPS)
    rda.rda_mla_append_q4(kv.to(dev), cache, table.to(dev), torch.tensor(after, dtype=torch.int32, device=dev),
                          torch.tensor(cu, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert torch.equal(cache.cpu(), want)


def check_read(cache, table, lens, cu, total, stride=None):
    dev = cache.device
    go = guarded((total, stride or 576), torch.bfloat16, dev)
    go.t.fill_(7.0)
    out = go.t[:, :576]
    before = out.clone()
    got = rda.rda_mla_read_q4(cache, table.to(dev), lens, total,
                              None if cu is None else torch.tensor(cu, dtype=torch.int32, device=dev), out=out)
    torch.cuda.synchronize()
    go.check("out")
    if stride:
        assert bool((go.t[:, 576:] == 7.0).all())
    each = total // table.shape[0]
    want = ref.read(cache.cpu(), table, lens, cu or [each * i for i in range(table.shape[0] + 1)], total, before)
    got = got.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


@pytest.mark.parametrize("new,after,page,total,stride", [
    ([1], [1], 8, 1, None), ([65], [65], 64, 65, None), ([5, 0, 130, 1], [5, 20, 200, 64], 64, 136, None),
    ([3, 9], [40, 9], 16, 20, 640), ([2] * 130, [30] * 130, 32, 260, None)])
def test_read(dev, new, after, page, total, stride):
    """Every byte pattern of the codes, scales of all sizes; rows behind the last part stay."""
    say(f"[read q4] new={new[:8]} after={after[:8]} page={page}")
    table, pool = tables(after, page, 3)
    g = torch.Generator().manual_seed(4)
    cache = torch.randint(0, 256, (pool, page, 400), generator=g).to(torch.uint8)
    cache[..., 256:272] = torch.randint(7, 253, (pool, page, 16), generator=g).to(torch.uint8)
    cache[..., 256:272][torch.rand(pool, page, 16, generator=g) < 0.02] = 255
    cache[..., 272:] = torch.randn(pool, page, 64, generator=g).bfloat16().view(torch.uint8)
    lens = torch.tensor(after, dtype=torch.int32, device=dev)
    check_read(cache.to(dev), table, lens, offsets(new), total, stride)
    if len(set(new)) == 1 and total == sum(new):
        check_read(cache.to(dev), table, lens, None, total, stride)


def test_read_out_of_range(dev):
    """Zeros where a position or page id is out of range."""
    say("[read q4] out of range")
    g = torch.Generator().manual_seed(5)
    cache = torch.randint(0, 256, (3, 8, 400), generator=g).to(torch.uint8)
    cache[..., 256:272], cache[..., 272:] = 130, 0
    table = torch.tensor([[0, -1], [7, 2], [1, 1]], dtype=torch.int32)
    lens = torch.tensor([12, 16, 20], dtype=torch.int32, device=dev)
    check_read(cache.to(dev), table, lens, [0, 14, 24, 34], 34)


def test_no_rows(dev):
    cache = torch.zeros(2, 8, 400, dtype=torch.uint8, device=dev)
    table = torch.zeros(1, 2, dtype=torch.int32, device=dev)
    lens = torch.zeros(1, dtype=torch.int32, device=dev)
    assert rda.rda_mla_read_q4(cache, table, lens, 0).shape == (0, 576)
    rda.rda_mla_append_q4(torch.zeros(0, 576, dtype=torch.bfloat16, device=dev), cache, table, lens)
    empty = torch.zeros(0, 8, 400, dtype=torch.uint8, device=dev)
    kv = torch.ones(3, 576, dtype=torch.bfloat16, device=dev)
    rda.rda_mla_append_q4(kv, empty, table, lens + 3)
    assert float(rda.rda_mla_read_q4(empty, table, lens + 3, 3).abs().max()) == 0
    torch.cuda.synchronize()
    assert int(cache.max()) == 0


def test_back_and_forth(dev):
    """Values that came out of the cache go in again as the same values."""
    say("[append, read q4] back and forth")
    cache, table, lens, cu = append(dev, rows(90, 15), [40, 50], [40, 61], 16, norm_weight(6), seed=2)
    once = rda.rda_mla_read_q4(cache, table.to(dev), lens, 90, cu)
    rda.rda_mla_append_q4(once, cache, table.to(dev), lens, cu)
    again = rda.rda_mla_read_q4(cache, table.to(dev), lens, 90, cu)
    assert torch.equal(once, again)
