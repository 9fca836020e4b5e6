"""GPU tests of rda_mla_decode (absorbed latent attention over a paged cache,
with and without a shared prefix) and of rda_mla_append, against the plain
64-bit forms."""
import pytest
import torch

import mla_ref
from gated_delta_amd import rda
from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def make(dev, lens, T, H, page, seed, prefix=0, spread=1.0, spare=2, width=None):
    """Queries, a shuffled page pool whose unused rows are NaN, tables."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    npre = -(-prefix // page)
    pool = sum(need) + npre + spare
    cache = torch.full((pool, page, 576), float("nan"), dtype=torch.bfloat16)
    perm = torch.randperm(pool, generator=g).tolist()
    width = width or max(1, max(need, default=1))
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0

    def fill(n):
        nonlocal at
        pages = perm[at:at + -(-n // page)]
        at += len(pages)
        rows = torch.randn(n, 576, generator=g).bfloat16()
        for i, p in enumerate(pages):
            part = rows[i * page:(i + 1) * page]
            cache[p, :part.shape[0]] = part
        return pages

    for b, n in enumerate(lens):
        pages = fill(n)
        table[b, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
    pre = torch.tensor(fill(prefix), dtype=torch.int32) if prefix else None
    q = (spread * torch.randn(len(lens), T, H, 576, generator=g)).bfloat16()
    return (q.to(dev), cache.to(dev), table.to(dev),
            torch.tensor(lens, dtype=torch.int32, device=dev), None if pre is None else pre.to(dev))


def run(dev, lens, T, H, page, seed=0, prefix=0, spread=1.0):
    say(f"[mla decode] lens={lens if len(lens) < 12 else len(lens)} T={T} H={H} page={page} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, page, seed, prefix, spread)
    o, lse = rda.rda_mla_decode(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=prefix,
                                want_lse=True)
    torch.cuda.synchronize()
    ro, rl, bo, bl = mla_ref.decode(q.cpu(), cache.cpu(), table.cpu(), lens, SCALE,
                                    None if pre is None else pre.cpu(), prefix)
    mla_ref.check("o", o, ro, bo)
    mla_ref.check("lse", lse, rl, bl)
    return o, lse


@pytest.mark.parametrize("n", [1, 2, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 1100])
def test_one_sequence(dev, n):
    run(dev, [n], 1, 4, 64, seed=n)


@pytest.mark.parametrize("H", [1, 3, 16, 32, 33, 40, 64, 96, 128])
def test_head_counts(dev, H):
    run(dev, [97, 5], 1, H, 32, seed=H)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 40, 64])
def test_new_tokens(dev, T):
    """Each new token sees one row more than the one before."""
    run(dev, [T, T + 31, 150, T + 1], T, 3, 16, seed=T)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 256])
def test_pages(dev, page):
    run(dev, [1, page - 1, page, page + 1, 3 * page + 5], 2, 5, page, seed=page)


def test_rows_that_see_nothing(dev):
    """Empty sequences, and first tokens of sequences shorter than the step."""
    o, lse = run(dev, [0, 1, 2, 70, 0], 3, 4, 16, seed=1)
    assert not o[0].any() and not o[1, 0].any() and bool((lse[0] == float("-inf")).all())
    run(dev, [0, 0], 1, 4, 16, seed=1)


def test_many_ragged_sequences(dev):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 200, (300,), generator=g).tolist()
    run(dev, lens, 1, 2, 16, seed=2)


@pytest.mark.parametrize("lens,T,H,prefix", [
    ([5], 1, 4, 1), ([3, 40], 1, 4, 33), ([1, 2, 3, 4, 5, 6, 7, 8, 9], 1, 32, 700),
    ([0, 9], 2, 5, 64), ([20, 0, 64], 3, 40, 129), ([7] * 5, 4, 16, 2000),
])
def test_prefix(dev, lens, T, H, prefix):
    run(dev, lens, T, H, 32, seed=prefix, prefix=prefix)


def test_prefix_alone(dev):
    """No rows of their own: every query sees the prefix only."""
    q, cache, table, kl, pre = make(dev, [0, 0], 1, 4, 16, 4, prefix=50)
    o, _ = rda.rda_mla_decode(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=50)
    ro, _, bo, _ = mla_ref.decode(q.cpu(), cache.cpu(), table.cpu(), [0, 0], SCALE, pre.cpu(), 50)
    mla_ref.check("o", o, ro, bo)


def test_large_scores(dev):
    run(dev, [400, 33], 2, 8, 32, seed=5, spread=40.0)


def test_growing_scores(dev):
    """The running maximum moves in every tile by more than is tolerated
    without rescaling, and the key waves' maxima differ."""
    q, cache, table, kl, _ = make(dev, [900], 1, 4, 64, 6)
    q.fill_(1)
    for i in range(900):
        cache[int(table[0, i // 64]), i % 64, 512:] = i * 0.02
    o, lse = rda.rda_mla_decode(q, cache, table, kl, SCALE * 10, want_lse=True)
    ro, rl, bo, bl = mla_ref.decode(q.cpu(), cache.cpu(), table.cpu(), [900], SCALE * 10)
    mla_ref.check("o", o, ro, bo)
    mla_ref.check("lse", lse, rl, bl)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_in_masked_places(dev, bad):
    """The last new token's row holds infinities or NaN: the tokens before it
    do not see it (rows behind the last one are NaN in every test here)."""
    lens, T = [100, 64, 33], 3
    q, cache, table, kl, _ = make(dev, lens, T, 4, 16, 7)
    for b, n in enumerate(lens):
        cache[int(table[b, (n - 1) // 16]), (n - 1) % 16, ::7] = bad
    o, lse = rda.rda_mla_decode(q, cache, table, kl, SCALE, want_lse=True)
    torch.cuda.synchronize()
    ro, rl, bo, bl = mla_ref.decode(q.cpu(), cache.cpu(), table.cpu(), lens, SCALE)
    mla_ref.check("o", o[:, :2], ro[:, :2], bo[:, :2])
    mla_ref.check("lse", lse[:, :2], rl[:, :2], bl[:, :2])
    assert not torch.isfinite(o[:, 2, :, 0].float()).any()


def test_same_page_twice(dev):
    """One page listed twice, and two sequences on the same pages."""
    q, cache, table, kl, _ = make(dev, [64, 64], 1, 4, 16, 8)
    table[0, 2] = table[0, 1]
    table[1] = table[0]
    o, lse = rda.rda_mla_decode(q, cache, table, kl, SCALE, want_lse=True)
    ro, rl, bo, bl = mla_ref.decode(q.cpu(), cache.cpu(), table.cpu(), [64, 64], SCALE)
    mla_ref.check("o", o, ro, bo)


def test_far_pages(dev):
    """Pages beyond 32 bits of elements, and pages apart from each other."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB of GPU memory")
    q, cache, table, kl, _ = make(dev, [200, 90], 1, 8, 64, 9)
    a, _ = rda.rda_mla_decode(q, cache, table, kl, SCALE)
    big = torch.empty(70000, 64, 576, dtype=torch.bfloat16, device=dev)
    shift = 70000 - cache.shape[0]
    big[shift:] = cache
    far = torch.where(table >= 0, table + shift, table)
    b, _ = rda.rda_mla_decode(q, big, far, kl, SCALE)
    assert torch.equal(a, b)
    # pages interleaved with those of other layers
    pool = big[:4 * cache.shape[0]].view(cache.shape[0], 4, 64, 576)
    pool[:, 2] = cache
    c, _ = rda.rda_mla_decode(q, pool[:, 2], table, kl, SCALE)
    assert torch.equal(a, c)


def test_bad_pages_stay_in_bounds(dev):
    q, cache, table, kl, _ = make(dev, [64, 64], 1, 4, 16, 10)
    table[0, 1], table[1, 2] = 1 << 30, -7
    kl[1] = 1 << 30
    rda.rda_mla_decode(q, cache, table, kl, SCALE)
    kl[0] = -3
    o, _ = rda.rda_mla_decode(q, cache, table, kl, SCALE)
    torch.cuda.synchronize()
    assert not o[0].any()


def test_deterministic(dev):
    lens = [1000, 3, 500, 777]
    q, cache, table, kl, pre = make(dev, lens, 3, 32, 64, 11, prefix=200)
    a = rda.rda_mla_decode(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=200, want_lse=True)
    for _ in range(3):
        b = rda.rda_mla_decode(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=200, want_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_replays_with_new_lengths(dev):
    """A captured call reads lengths, tables and rows when it is replayed."""
    lens = [300, 40]
    q, cache, table, kl, _ = make(dev, lens, 2, 32, 32, 12, width=12)
    ws = torch.empty(rda.rda_mla_decode_workspace_bytes(2, 2, 32), dtype=torch.uint8, device=dev)
    o = torch.empty(2, 2, 32, 512, dtype=torch.bfloat16, device=dev)
    rda.rda_mla_decode(q, cache, table, kl, SCALE, o=o, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rda.rda_mla_decode(q, cache, table, kl, SCALE, o=o, workspace=ws)
    for new in ([300, 40], [20, 33], [299, 2], [0, 7]):
        kl.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want, _ = rda.rda_mla_decode(q, cache, table, kl, SCALE)
        assert torch.equal(o, want)


def test_two_streams_two_workspaces(dev):
    q, cache, table, kl, _ = make(dev, [700, 300], 1, 32, 64, 13)
    want, _ = rda.rda_mla_decode(q, cache, table, kl, SCALE)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [rda.rda_mla_decode(q, cache, table, kl, SCALE, o=torch.empty_like(want), stream=s)[0]
            for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)


def bound_append(ref):
    # fp32 arithmetic (sum of 512 squares, a root, two products: below 2^-14
    # relative) and one rounding to bf16
    return ref.abs() * (mla_ref.BF16_HALF_STEP + 2.0 ** -14) + 1e-38


@pytest.mark.parametrize("new,cached,page,norm", [
    ([1], [0], 16, True), ([1, 1, 1], [5, 15, 16], 16, True), ([3, 3], [14, 0], 16, False),
    ([5, 0, 40, 1], [0, 3, 7, 63], 32, True), ([100], [0], 64, True), ([2] * 70, [9] * 70, 8, True),
])
def test_append(dev, new, cached, page, norm):
    lens = [a + b for a, b in zip(new, cached)]
    _, cache, table, kl, _ = make(dev, lens, 1, 1, page, sum(new))
    cache = cache.nan_to_num(0.5)
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(sum(new), 640, generator=g).bfloat16().to(dev)
    kv = wide[:, 64:]
    weight = (1 + 0.1 * torch.randn(512, generator=g)).to(dev) if norm else None
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    ref = mla_ref.append(kv, cache, table.cpu(), lens, cu, weight, 1e-5)
    before = cache.clone()
    out = rda.rda_mla_append(kv, cache, table, kl, cu, weight=weight, eps=1e-5)
    torch.cuda.synchronize()
    assert out is cache
    mla_ref.check("cache", cache, ref, bound_append(ref))
    same = ref == before.cpu().double()     # rows that the call has to leave
    assert torch.equal(cache.cpu()[same], before.cpu()[same])
    if len(set(new)) == 1 and new[0]:
        again = rda.rda_mla_append(kv, before, table, kl, weight=weight, eps=1e-5)
        assert torch.equal(again, cache)


def test_append_zero_rows_and_extremes(dev):
    """A row of zeros stays zero; large and tiny rows stay finite."""
    _, cache, table, kl, _ = make(dev, [4], 1, 1, 8, 0)
    kv = torch.zeros(4, 576, dtype=torch.bfloat16, device=dev)
    kv[1], kv[2], kv[3] = 1e15, 1e-30, -1e15
    rda.rda_mla_append(kv, cache, table, kl, weight=torch.ones(512, device=dev), eps=1e-5)
    rows = cache[int(table[0, 0]), :4].float()
    assert not rows[0].any() and torch.isfinite(rows).all()
    assert torch.equal(rows[1, :512], torch.ones(512, device=dev))


def test_append_out_of_range_writes_nothing(dev):
    _, cache, table, kl, _ = make(dev, [40, 8], 1, 1, 8, 0)
    cache = cache.nan_to_num(0.25)
    before = cache.clone()
    kv = torch.ones(2, 576, dtype=torch.bfloat16, device=dev)
    table[0, 4], table[1, 0] = 1 << 29, -1
    rda.rda_mla_append(kv, cache, table, kl, eps=0.0)
    kl[0], kl[1] = 0, 1 << 30
    rda.rda_mla_append(kv, cache, table, kl, eps=0.0)
    torch.cuda.synchronize()
    assert torch.equal(cache, before)


def test_append_then_decode(dev):
    """The rows that append writes are the rows that decode reads."""
    B, T, H, page = 3, 2, 32, 16
    lens = [20, 2, 49]
    q, cache, table, kl, _ = make(dev, lens, T, H, page, 14)
    kv = torch.randn(B * T, 576, device=dev).bfloat16()
    weight = torch.rand(512, device=dev) + 0.5
    rda.rda_mla_append(kv, cache, table, kl, weight=weight)
    o, lse = rda.rda_mla_decode(q, cache, table, kl, SCALE, want_lse=True)
    ro, rl, bo, bl = mla_ref.decode(q.cpu(), cache.cpu(), table.cpu(), lens, SCALE)
    mla_ref.check("o", o, ro, bo)
    mla_ref.check("lse", lse, rl, bl)
