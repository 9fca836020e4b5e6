"""GPU tests of rda_mla_prefill at batches long enough for its kernel of 256
queries a workgroup, against the plain 64-bit form on the rows and heads where
blocks begin and end, and against the same sequences in small calls."""
import pytest
import torch

import mla_ref
from gated_delta_amd import rda
from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
EDGES = (0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 255, 256, 257, 511, 512)


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def make(dev, lq, lk, H, seed, spread=2.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    q = (spread * torch.randn(sum(lq), H, 192, generator=g, device=dev)).bfloat16()
    kv = torch.randn(sum(lk), H, 256, generator=g, device=dev).bfloat16()
    rows = torch.randn(sum(lk), 576, generator=g, device=dev).bfloat16()
    return q, kv, rows[:, 512:]


def compare(o, lse, q, kv, pe, lq, lk, causal, heads, scale=SCALE, rows=None):
    o, lse = o.cpu(), lse.cpu()
    q, kv, pe = q.cpu(), kv.cpu(), pe.cpu()
    cq, ck = offsets(lq), offsets(lk)
    for n, (a, c) in enumerate(zip(cq[:-1], ck[:-1])):
        if not lq[n]:
            continue
        at = sorted({i for e in EDGES for i in (e, lq[n] - 1 - e) if 0 <= i < lq[n]}) if rows is None else rows
        limit = [i + 1 + lk[n] - lq[n] if causal else lk[n] for i in at]
        for h in heads:
            k = torch.cat([kv[c:c + lk[n], h, :128], pe[c:c + lk[n]]], 1)
            ro, rl, bo, bl = mla_ref.attend(q[a:a + lq[n], h][at], k, kv[c:c + lk[n], h, 128:], scale, limit)
            mla_ref.check(f"o {n} {h}", o[a:a + lq[n], h][at], ro, bo)
            mla_ref.check(f"lse {n} {h}", lse[a:a + lq[n], h][at], rl, bl)


@pytest.mark.parametrize("lq,lk,H", [
    ([1000], [2050], 128),                       # queries behind cached keys
    ([2049], [2049], 64),
    ([2300, 0, 1, 1500, 257], [2300, 3000, 1, 1800, 3400], 48),
    ([3000, 511], [60, 4100], 40),               # rows that see nothing
    ([8192], [8192], 16),
])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_and_heads(dev, lq, lk, H, causal):
    say(f"[mla prefill wide] lq={lq} lk={lk} H={H} causal={causal}")
    q, kv, pe = make(dev, lq, lk, H, sum(lq) + H)
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, offsets(lq), offsets(lk), causal=causal, want_lse=True)
    torch.cuda.synchronize()
    compare(o, lse, q, kv, pe, lq, lk, causal, (0, H - 1))


def test_no_keys(dev):
    """Sequences without keys beside one that has them all."""
    lq, lk = [1000, 600], [4200, 0]
    q, kv, pe = make(dev, lq, lk, 80, 1)
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, offsets(lq), offsets(lk), want_lse=True)
    assert not o[1000:].any() and bool((lse[1000:] == float("-inf")).all())
    assert bool(torch.isfinite(lse[:1000]).all())


@pytest.mark.parametrize("spread", [0.0, 60.0])
def test_large_scores(dev, spread):
    q, kv, pe = make(dev, [2100], [2100], 64, 3, spread)
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, want_lse=True)
    compare(o, lse, q, kv, pe, [2100], [2100], True, (0, 63))


def test_growing_scores(dev):
    """The running reference moves in many steps."""
    T, H = 2100, 64
    q, kv, pe = make(dev, [T], [T], H, 5)
    q, pe = q * 0 + 1, pe * 0
    kv[:, :, :128] = (torch.arange(T, device=dev).float() * 0.01).bfloat16()[:, None, None]
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE * 20, want_lse=True)
    compare(o, lse, q, kv, pe, [T], [T], True, (0,), scale=SCALE * 20)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_bad_values_in_masked_places(dev, bad):
    """A key row that holds infinities or NaN reaches only the queries that see
    it, whatever part of a block it lies in."""
    T, H = 2300, 64
    for at in (100, 255, 256, 1311, 2299):
        q, kv, pe = make(dev, [T], [T], H, 6)
        clean, _ = rda.rda_mla_prefill(q, kv, pe, SCALE)
        kv[at, 1] = bad
        kv[at, 2, 128 + 7] = bad
        o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, want_lse=True)
        # (products of a block with such a value are taken in another order)
        part = {0: slice(0, T), 1: slice(0, at), 2: slice(0, at)}
        for h, rows in part.items():
            assert bool(torch.isfinite(o[rows, h].float()).all()), (at, h)
        near = [i for i in (0, at - 70, at - 33, at - 1) if 0 <= i < at]
        compare(o, lse, q, kv, pe, [T], [T], True, (1, 2), rows=near)
        assert torch.equal(o[:, 0], clean[:, 0]) and torch.equal(o[:, 3:], clean[:, 3:])
        assert not bool(torch.isfinite(o[at:, 1].float()).any()) or bad == float("-inf")
        assert not bool(torch.isfinite(o[at:, 2, 7].float()).any())
        assert bool(torch.isfinite(o[at:, 2, 8:].float()).all())


def test_strides(dev):
    """Wider rows, one of them a power of two and one not a multiple of 16."""
    T, H = 2100, 64
    q, kv, pe = make(dev, [T], [T], H, 8)
    wq = torch.full((T, H * 192 + 24), 7.0, dtype=torch.bfloat16, device=dev)
    wk = torch.full((T, 1 << 15), 7.0, dtype=torch.bfloat16, device=dev)
    wq[:, 8:8 + H * 192] = q.reshape(T, -1)
    wk[:, 64:64 + H * 256] = kv.reshape(T, -1)
    a, _ = rda.rda_mla_prefill(q, kv, pe.contiguous(), SCALE)
    b, _ = rda.rda_mla_prefill(wq[:, 8:8 + H * 192].unflatten(1, (H, 192)),
                               wk[:, 64:64 + H * 256].unflatten(1, (H, 256)), pe, SCALE)
    assert torch.equal(a, b)


def test_offsets_out_of_range_stay_in_bounds(dev):
    """Device offsets are trusted, but never used out of bounds."""
    q, kv, pe = make(dev, [2100], [2100], 64, 11)
    for cu in ([0, 1 << 30], [-5, 2100], [1900, 10], [1 << 30, -(1 << 30)]):
        t = torch.tensor(cu, dtype=torch.int32, device=dev)
        rda.rda_mla_prefill(q, kv, pe, SCALE, t, t)
    torch.cuda.synchronize()


def test_rows_behind_the_last_sequence_stay(dev):
    """Output rows that belong to no sequence keep what they held."""
    T, H = 2300, 64
    q, kv, pe = make(dev, [T], [T], H, 12)
    o = torch.full((T, H, 128), 3.0, dtype=torch.bfloat16, device=dev)
    t = torch.tensor([0, 2100], dtype=torch.int32, device=dev)
    rda.rda_mla_prefill(q, kv, pe, SCALE, t, t, o=o)
    want, _ = rda.rda_mla_prefill(q[:2100], kv[:2100], pe[:2100], SCALE)
    assert torch.equal(o[:2100], want) and bool((o[2100:] == 3).all())


@pytest.mark.parametrize("T,H", [(300, 4), (2100, 64)])
def test_captured_and_replayed(dev, T, H):
    """A captured call follows its inputs and offsets from replay to replay,
    between eager calls of the same kernels."""
    q, kv, pe = make(dev, [T], [T], H, 13)
    cu = torch.tensor([0, T], dtype=torch.int32, device=dev)
    o, lse = torch.empty(T, H, 128, dtype=torch.bfloat16, device=dev), torch.empty(T, H, device=dev)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        rda.rda_mla_prefill(q, kv, pe, SCALE, cu, cu, o=o, lse=lse, want_lse=True)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            rda.rda_mla_prefill(q, kv, pe, SCALE, cu, cu, o=o, lse=lse, want_lse=True)
    for n in range(3):
        q.copy_(make(dev, [T], [T], H, 20 + n)[0])
        cu[1] = T - 40 * n
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, wl = rda.rda_mla_prefill(q, kv, pe, SCALE, cu, cu, want_lse=True)
        m = T - 40 * n
        assert torch.equal(o[:m], want[:m]) and torch.equal(lse[:m], wl[:m])
