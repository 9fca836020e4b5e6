"""GPU tests of rda_mla_prefill (expanded latent attention) against the plain
64-bit form, at the sizes, masks and values where a tiled kernel goes wrong."""
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


def offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def make(dev, lq, lk, H, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    q = (spread * torch.randn(sum(lq), H, 192, generator=g)).bfloat16()
    kv = torch.randn(sum(lk), H, 256, generator=g).bfloat16()
    rows = torch.randn(sum(lk), 576, generator=g).bfloat16()
    return q.to(dev), kv.to(dev), rows.to(dev)[:, 512:]


def run(dev, lq, lk, H, causal, seed=0, spread=2.0, scale=SCALE):
    say(f"[mla prefill] lq={lq} lk={lk} H={H} causal={causal}")
    q, kv, pe = make(dev, lq, lk, H, seed, spread)
    cq, ck = offsets(lq), offsets(lk)
    o, lse = rda.rda_mla_prefill(q, kv, pe, scale, cq, ck, causal=causal, want_lse=True)
    torch.cuda.synchronize()
    ro, rl, bo, bl = mla_ref.prefill(q.cpu(), kv.cpu(), pe.cpu(), scale, cq, ck, causal)
    mla_ref.check("o", o, ro, bo)
    mla_ref.check("lse", lse, rl, bl)
    return o, lse


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 321])
@pytest.mark.parametrize("causal", [True, False])
def test_one_sequence(dev, T, causal):
    run(dev, [T], [T], 2, causal, seed=T)


@pytest.mark.parametrize("H", [1, 3, 16, 40])
def test_head_counts(dev, H):
    run(dev, [70], [70], H, True, seed=H)


@pytest.mark.parametrize("lq,lk", [
    ([1], [300]), ([5], [64]), ([130], [131]), ([3, 1, 200], [70, 1, 200]),
    ([0, 5, 0, 129, 0], [3, 5, 0, 200, 64]),      # empty sequences, keys without queries
    ([10], [4]), ([140], [5]), ([33, 66], [0, 60]),  # rows that see nothing
    ([1] * 9, [1, 2, 63, 64, 65, 127, 128, 129, 0]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_packed(dev, lq, lk, causal):
    o, lse = run(dev, lq, lk, 3, causal, seed=len(lq) + sum(lq))


def test_no_keys(dev):
    q, kv, pe = make(dev, [7], [0], 2, 0)
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, [0, 7], [0, 0], want_lse=True)
    assert not o.any() and bool((lse == float("-inf")).all())


def test_no_queries(dev):
    q, kv, pe = make(dev, [0], [5], 2, 0)
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, [0, 0], [0, 5], want_lse=True)
    assert o.shape == (0, 2, 128)


def test_large_scores(dev):
    """Scores far apart (nearly one-hot rows) and far from zero."""
    run(dev, [150], [150], 2, True, seed=3, spread=60.0)
    run(dev, [150], [150], 2, True, seed=4, spread=0.0)


def test_growing_scores(dev):
    """Keys whose scores grow along the sequence: the running maximum moves in
    every tile, by more than the kernel tolerates without rescaling."""
    T, H = 500, 1
    q, kv, pe = make(dev, [T], [T], H, 5)
    q = q * 0 + 1
    ramp = torch.arange(T, device=dev).float()[:, None] * 0.01
    kv[:, 0, :128] = ramp.bfloat16()
    o, lse = rda.rda_mla_prefill(q, kv, pe * 0, SCALE * 20, causal=True, want_lse=True)
    ro, rl, bo, bl = mla_ref.prefill(q.cpu(), kv.cpu(), (pe * 0).cpu(), SCALE * 20, [0, T], [0, T], True)
    mla_ref.check("o", o, ro, bo)
    mla_ref.check("lse", lse, rl, bl)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_bad_values_in_masked_places(dev, bad):
    """A key row that holds infinities or NaN reaches only the queries that
    see it; neighbouring sequences not at all."""
    lq, at = [40, 200, 30], 150       # row 150 of the middle sequence
    q, kv, pe = make(dev, lq, lq, 2, 6)
    cq = offsets(lq)
    kv[40 + at, 1] = bad
    kv[40 + 199, 0, 128:] = bad        # values only, the last key
    pe = pe.clone()
    o, lse = rda.rda_mla_prefill(q, kv, pe, SCALE, cq, want_lse=True)
    torch.cuda.synchronize()
    ro, rl, bo, bl = mla_ref.prefill(q.cpu(), kv.cpu(), pe.cpu(), SCALE, cq, cq, True)
    clean = torch.ones(sum(lq), 2, dtype=torch.bool)
    clean[40 + at:240, 1] = False
    clean[239, 0] = False
    mla_ref.check("o", o.cpu()[clean], ro[clean], bo[clean])
    mla_ref.check("lse", lse.cpu()[clean], rl[clean], bl[clean])
    assert not torch.isfinite(o.cpu()[239, 0].float()).any()


def test_finite_values_beside_bad_ones(dev):
    """In a tile with an infinite value, every query's other channels and the
    queries that do see it are as the formula has them."""
    T = 90
    q, kv, pe = make(dev, [T], [T], 1, 7)
    kv[70, 0, 128 + 5] = float("inf")
    o, _ = rda.rda_mla_prefill(q, kv, pe, SCALE)
    kv2 = kv.clone()
    kv2[70, 0, 128 + 5] = 0
    ro, _, bo, _ = mla_ref.prefill(q.cpu(), kv2.cpu(), pe.cpu(), SCALE, [0, T], [0, T], True)
    ro[70:, 0, 5] = float("inf")
    mla_ref.check("o", o, ro, bo)


def test_strides(dev):
    """q, kv and k_pe as slices of wider rows."""
    T, H = 133, 2
    q, kv, pe = make(dev, [T], [T], H, 8)
    wq = torch.full((T, H * 192 + 24), 7.0, dtype=torch.bfloat16, device=dev)
    wk = torch.full((T, H * 256 + 640), 7.0, dtype=torch.bfloat16, device=dev)
    wq[:, 8:8 + H * 192] = q.reshape(T, -1)
    wk[:, 64:64 + H * 256] = kv.reshape(T, -1)
    q2 = wq[:, 8:8 + H * 192].unflatten(1, (H, 192))
    k2 = wk[:, 64:64 + H * 256].unflatten(1, (H, 256))
    a, _ = rda.rda_mla_prefill(q, kv, pe.contiguous(), SCALE)
    b, _ = rda.rda_mla_prefill(q2, k2, pe, SCALE)
    assert torch.equal(a, b)


def test_far_rows(dev):
    """Key rows further apart than 32 bits of elements."""
    T, H, stride = 300, 1, 1 << 23
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB of GPU memory")
    q, kv, pe = make(dev, [T], [T], H, 9)
    wide = torch.empty((T - 1) * stride + 256, dtype=torch.bfloat16, device=dev)
    far = torch.as_strided(wide, (T, H, 256), (stride, 256, 1))
    far.copy_(kv)
    a, _ = rda.rda_mla_prefill(q, kv, pe, SCALE)
    b, _ = rda.rda_mla_prefill(q, far, pe, SCALE)
    assert torch.equal(a, b)


def test_deterministic_and_packed_alone(dev):
    """A sequence's result does not depend on the batch it is packed in."""
    lq = [130, 77, 300]
    q, kv, pe = make(dev, lq, lq, 4, 10)
    cq = offsets(lq)
    o, _ = rda.rda_mla_prefill(q, kv, pe, SCALE, cq)
    again, _ = rda.rda_mla_prefill(q, kv, pe, SCALE, torch.tensor(cq, dtype=torch.int32, device=dev))
    assert torch.equal(o, again)
    for a, b in zip(cq, cq[1:]):
        alone, _ = rda.rda_mla_prefill(q[a:b], kv[a:b], pe[a:b], SCALE)
        assert torch.equal(alone, o[a:b])


def test_offsets_out_of_range_stay_in_bounds(dev):
    """Device offsets are trusted, but never used out of bounds."""
    q, kv, pe = make(dev, [100], [100], 2, 11)
    for cu in ([0, 1 << 30], [-5, 100], [90, 10], [1 << 30, -(1 << 30)]):
        t = torch.tensor(cu, dtype=torch.int32, device=dev)
        rda.rda_mla_prefill(q, kv, pe, SCALE, t, t)
    torch.cuda.synchronize()


def test_other_stream(dev):
    q, kv, pe = make(dev, [200], [200], 4, 12)
    a, _ = rda.rda_mla_prefill(q, kv, pe, SCALE)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, _ = rda.rda_mla_prefill(q, kv, pe, SCALE, o=torch.empty_like(a), stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
