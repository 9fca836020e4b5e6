"""GPU tests of rda_mla_decode_q4 over batches whose tiles are shared out in
different ways, caches of hundreds of thousands of rows, pages apart, lengths
and page ids out of range, and the same bits from the same call."""
import pytest
import torch

import mla_q4_ref as ref
from gated_delta_amd import rda
from gpu_util import guarded, need_gpu, say
from test_gpu_mla_decode_q4 import SCALE, compare, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def spread(n, low, high, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, high + 1, (n,), generator=g).tolist()


@pytest.mark.parametrize("lens,T,H", [
    (spread(60, 300, 900, 1), 1, 8),       # shares end with the sequence, some hold several
    (spread(120, 1, 120, 2), 2, 8),        # whole sequences
    (spread(8, 255, 284, 3), 5, 16),       # short shares, few sequences
    ([0, 0, 700, 0, 33, 1] * 8, 3, 24),    # empty ones between, two blocks of rows
    (spread(250, 1, 40, 4), 1, 8),         # nearly as many sequences as workgroups
    (spread(250, 40, 300, 4), 1, 4),       # more shares than workgroups: equal shares
    (spread(300, 0, 90, 5), 1, 4),         # more sequences than a workgroup has threads
    (spread(600, 0, 90, 5), 1, 1),         # and than workgroups
    ([5000] + [1] * 30, 1, 8),             # one long, many short
    (spread(40, 1, 200, 6), 5, 32),        # three blocks of 64 rows a sequence
    ([1] * 3, 1, 40), ([31, 32, 33, 64, 65], 1, 65),
    (spread(64, 1, 300, 9), 1, 8),         # as many sequences as a wave plans by itself
    (spread(65, 1, 300, 9), 1, 8),
    (spread(64, 1500, 2500, 10), 1, 2),    # longer shares: two workgroups a CU
    (spread(2, 2000, 4000, 11), 1, 32),    # 64 query rows with many pieces each, joined by 16 waves
    (spread(5, 900, 2000, 12), 1, 13),     # 65 of them: by 4
    (spread(16, 900, 2000, 13), 1, 32),    # 512
    (spread(19, 900, 2000, 14), 1, 27),    # 513: by one
])
def test_shares(dev, lens, T, H):
    run(dev, lens, T, H, 32, seed=len(lens) + T)


@pytest.mark.parametrize("lens,T,H,prefix", [
    ([17, 33, 0, 1] * 6, 1, 40, 11),       # a prefix of less than a tile, many blocks
    ([5, 2] * 9, 3, 16, 70),
    (spread(20, 0, 60, 7), 8, 120, 40),    # many rows of a short prefix
    ([40, 3], 1, 64, 700),                 # 64 rows a sequence, the prefix for 32 at a time
    (spread(130, 1, 50, 8), 1, 32, 2100),   # 32 rows a sequence, the prefix for 64 at a time
    ([0, 0], 2, 3, 33),
    ([9] * 16, 1, 32, 5000),               # equal pieces of each block of query rows
    ([9] * 33, 1, 40, 1100),               # blocks of 64 rows, which cross sequences
    ([70, 0, 3], 1, 5, 2000),              # few rows: short pieces
])
def test_prefixes(dev, lens, T, H, prefix):
    run(dev, lens, T, H, 16, seed=len(lens) + T, prefix=prefix)


@pytest.mark.parametrize("lens,T,H,page,prefix", [
    ([262144], 1, 2, 64, 0),
    ([200003, 7, 4099], 1, 2, 256, 0),
    ([131075], 2, 2, 16, 0),
    ([90, 1], 1, 2, 64, 262001),
    ([66000], 3, 48, 128, 0),              # 144 query rows: each is joined by one wave
])
def test_long(dev, lens, T, H, page, prefix):
    """Queries spread so that a few rows hold most of the weight: the outputs are
    then far larger than the bound, which grows with the number of rows."""
    say(f"[mla q4] long: lens={lens} T={T} H={H} page={page} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, page, 20 + T + page, prefix, spread=2.0)
    o, lse = compare(q, cache, table, kl, pre, prefix, lens)


@pytest.mark.parametrize("page,apart", [(8, 16), (64, 400 * 64), (16, 1 << 20), (1 << 16, 0)])
def test_pages_apart(dev, page, apart):
    """Pages that lie in a larger allocation, what is between them NaN."""
    say(f"[mla q4] pages of {page} rows, {apart} bytes between")
    lens = [70, 0, 133]
    q, cache, table, kl, _ = make(dev, lens, 2, 5, page, 4)
    n = cache.shape[0]
    step = page * 400 + apart
    pool = torch.full((n * step,), 255, dtype=torch.uint8, device=dev)
    wide = pool.as_strided((n, page, 400), (step, 400, 1))
    wide.copy_(cache)
    compare(q, wide, table, kl, None, 0, lens)


def test_far_pages(dev):
    """A cache of more than 2^32 bytes: pages behind that distance."""
    say("[mla q4] far pages")
    lens, page = [100, 40], 64
    q, cache, table, kl, _ = make(dev, lens, 1, 8, page, 5, spare=0)
    far = torch.empty((1 << 32) // (page * 400) + 8, page, 400, dtype=torch.uint8, device=dev)
    n = cache.shape[0]
    far[-n:] = cache
    o, _ = rda.rda_mla_decode_q4(q, far, table + (far.shape[0] - n), kl, SCALE)
    want, _ = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE)
    assert torch.equal(o, want)
    rows = torch.randn(140, 576, device=dev).bfloat16()
    cu = torch.tensor([0, 100, 140], dtype=torch.int32, device=dev)
    rda.rda_mla_append_q4(rows, far, table + (far.shape[0] - n), kl, cu)
    rda.rda_mla_append_q4(rows, cache, table, kl, cu)
    assert torch.equal(far[-n:], cache)
    assert torch.equal(rda.rda_mla_read_q4(far, table + (far.shape[0] - n), kl, 140, cu),
                       rda.rda_mla_read_q4(cache, table, kl, 140, cu))


def test_lengths_and_ids_out_of_range(dev):
    """Lengths are clamped to what the table holds; ids out of range read some page,
    and the sequences beside theirs keep their values."""
    say("[mla q4] lengths and ids out of range")
    lens = [48, 20, 48, 30, 0]
    q, cache, table, kl, _ = make(dev, lens, 1, 6, 16, 6, width=3)
    want = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, want_lse=True)
    kl2 = kl.clone()
    kl2[0], kl2[2], kl2[4] = 2 ** 31 - 1, 49, -7
    t2 = table.clone()
    t2[3] = torch.tensor([2 ** 31 - 1, -2 ** 31, cache.shape[0]], dtype=torch.int32)
    go, gl = guarded((5, 1, 6, 512), torch.bfloat16, dev), guarded((5, 1, 6), torch.float32, dev)
    rda.rda_mla_decode_q4(q, cache, t2, kl2, SCALE, o=go.t, lse=gl.t)
    torch.cuda.synchronize()
    go.check("o")
    gl.check("lse")
    keep = [0, 1, 2, 4]
    assert torch.equal(go.t[keep], want[0][keep]) and torch.equal(gl.t[keep], want[1][keep])


def test_no_pages(dev):
    q = torch.ones(2, 1, 3, 576, dtype=torch.bfloat16, device=dev)
    kl = torch.tensor([5, 0], dtype=torch.int32, device=dev)
    for cache, table in ((torch.empty(0, 8, 400, dtype=torch.uint8, device=dev), torch.zeros(2, 1, dtype=torch.int32, device=dev)),
                         (torch.zeros(2, 8, 400, dtype=torch.uint8, device=dev), torch.empty(2, 0, dtype=torch.int32, device=dev))):
        o, lse = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, want_lse=True)
        assert float(o.abs().max()) == 0 and bool(torch.isneginf(lse).all())
    o, _ = rda.rda_mla_decode_q4(q[:0], cache, table[:0], kl[:0], SCALE)
    assert o.shape == (0, 1, 3, 512)
    torch.cuda.synchronize()


@pytest.mark.parametrize("lens,T,H,prefix", [([777] * 3, 1, 32, 0), ([3000, 5], 2, 40, 0), ([50] * 70, 1, 32, 500)])
def test_same_bits(dev, lens, T, H, prefix):
    say(f"[mla q4] same bits B={len(lens)} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, 64, 8, prefix)
    kw = dict(prefix_table=pre, prefix_len=prefix, want_lse=True)
    want = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, **kw)
    for _ in range(10):
        got = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("scale", [1e-30, 1e-4, 1.0, 50.0])
def test_scales(dev, scale):
    """From all rows alike to one row alone."""
    say(f"[mla q4] scale={scale}")
    lens = [130, 33]
    q, cache, table, kl, _ = make(dev, lens, 1, 5, 16, 9, spread=0.1)
    o, lse = rda.rda_mla_decode_q4(q, cache, table, kl, scale, want_lse=True)
    ro, rl, bo, bl = ref.decode(q, cache, table.cpu(), lens, scale)
    ref.check("o", o, ro, bo)
    ref.check("lse", lse, rl, bl)


@pytest.mark.parametrize("size", [0.0, 1e-38, 1e-30, 1e20])
def test_query_magnitudes(dev, size):
    """Queries of zeros, subnormal numbers and very large ones, the last against rows
    scaled down as far."""
    say(f"[mla q4] queries of {size}")
    lens = [70]
    q, cache, table, kl, _ = make(dev, lens, 1, 3, 16, 10)
    q.copy_((q.float() * size).bfloat16())
    if size > 1:
        cache[..., 256:272] = torch.where(cache[..., 256:272] == 255, cache[..., 256:272], cache[..., 256:272] - 66)
        q[..., 512:] = 0
    o, lse = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, want_lse=True)
    ro, rl, bo, bl = ref.decode(q, cache, table.cpu(), lens, SCALE)
    ref.check("o", o, ro, bo)
    ref.check("lse", lse, rl, bl)
