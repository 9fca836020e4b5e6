"""GPU tests of rda_mla_decode_q4's scores, where the query's channels differ in
size: what the products with the codes may lose.

The matrix instruction adds eight products at a time, each cut towards zero to a
multiple of 2^-13 of the largest's power of two (the sum of its operands' exponents,
those of subnormal operands the format's least; 16384 random eights agree), and sums of
eight in 24 bits.  The kernel splits a query into hi + lo, 8-bit floats e4m3 (4 bits, last
step 2^-9), with hi's scale H for each 32 channels, whose largest magnitude M is
then below 3.875 H, and at least 1.9375 H.  hi is a whole multiple of 2^-9 H up to
3.75 H; with codes (multiples of 1/2, exponents up to 2) its products end at
2^-10, the largest exponent is 1 + 2: 2^-13 apart, nothing is cut.  hi leaves 2^-3 H
at most; lo has the scale 2^-11 H, so it is at most 256 and its products, with exponents
up to 8 + 2, are cut at multiples of 2^(10 - 13) 2^-11 H = 2^-14 H of the codes' unit or finer.

A channel of 2^-6 H (M / 64) or more has 4 bits in hi and 4 in lo, the last no less
than 2^-13 H, so its products end at 2^-14 H: exact.  A smaller one is hi in steps of
2^-9 H, which leave 2^-10 H at most, in 4 bits: off by 2^-15 H, and its product by
less than 2^-14 H units more.
"""
import pytest
import torch

import mla_q4_ref as ref
from gated_delta_amd import rda
from gpu_util import need_gpu, say
from mla_ref import BF16_HALF_STEP, LATENT
from test_gpu_mla_decode_q4 import SCALE, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.mark.parametrize("exponent", [0, 12])
@pytest.mark.parametrize("same_sign", [False, True])
@pytest.mark.parametrize("apart", [0, 14])
@pytest.mark.parametrize("H", [5, 40])
def test_exact_scores(dev, exponent, same_sign, apart, H):
    """One cached row, whose log-sum-exp is its score.  In four groups of 32 channels two
    of the query's are 1 and -1 and cancel against codes of 6, the others are 1/64 to 1/4
    with 8 bits: all are multiples of 2^-13, the codes of 1/2, and the sum of all
    magnitudes is below 2^8, so every sum of some of them has 22 bits and the score is exact.
    Groups are up to 2^14 apart, the query's and the rows' in opposite directions.  What is
    left: c = scale log2 e (two roundings), s c, times ln 2 (two), and a logarithm near that
    of 1; each 2^-24 relative, the last 2^-22."""
    say(f"[mla q4] exact scores, 2^{exponent}, groups 2^{apart} apart, H={H}")
    B, g = 24, torch.Generator().manual_seed(100 + H)
    shift = torch.randint(0, apart + 1, (B, 16), generator=g)
    rows = torch.zeros(B, 400, dtype=torch.uint8)
    rows[:, :256] = torch.randint(0, 256, (B, 256), generator=g, dtype=torch.int32).to(torch.uint8)
    rows[:, 256:272] = (127 + exponent + shift).to(torch.uint8)
    at = torch.arange(0, 16, 4) * 32 + torch.randint(0, 16, (4,), generator=g) * 2   # an even channel, and the next
    for c in at.tolist():
        rows[:, c // 2] = 0x77
    values = ref.values(rows)[:, None, None, :LATENT]
    q = torch.randint(128, 256, (B, 1, H, 512), generator=g) * 2.0 ** -13
    q *= 2.0 ** torch.randint(0, 4, (B, 1, H, 512), generator=g)
    q *= torch.where(values < 0, -1.0, 1.0) if same_sign else torch.randint(0, 2, q.shape, generator=g) * 2.0 - 1
    q[..., at], q[..., at + 1] = 1.0, -1.0
    q *= (2.0 ** -shift.double()).repeat_interleave(32, 1)[:, None, None]
    q = torch.cat([q, torch.zeros(B, 1, H, 64)], -1).bfloat16()
    products = q[..., :LATENT].double() * values
    assert float(products.abs().sum(-1).max()) < 256 * 2.0 ** exponent
    cache = torch.full((B, 8, 400), 255, dtype=torch.uint8)
    cache[:, 0] = rows
    table = torch.arange(B, dtype=torch.int32)[:, None].to(dev)
    lens = torch.ones(B, dtype=torch.int32, device=dev)
    o, lse = rda.rda_mla_decode_q4(q.to(dev), cache.to(dev), table, lens, SCALE, want_lse=True)
    want = SCALE * products.sum(-1)
    err = (lse.cpu().double() - want).abs()
    bound = 6 * 2.0 ** -24 * want.abs() + 2.0 ** -22
    assert bool((err <= bound).all()), (float((err / bound).max()), float(err.max()))
    assert torch.equal(o.cpu().double(), values.expand(B, 1, H, LATENT))


@pytest.mark.parametrize("lens,T,H", [([300, 40], 1, 6), ([777], 1, 32), ([90] * 12, 3, 24)])
@pytest.mark.parametrize("small", [2.0 ** -6, 2.0 ** -9, 2.0 ** -12])
def test_large_channels(dev, lens, T, H, small):
    """One channel of eight is 64 (so H = 32), with codes of 6 and -6 that cancel over the
    row; the others are small and all alike in sign."""
    say(f"[mla q4] large channels beside {small} lens={lens[:4]} T={T} H={H}")
    q, cache, table, kl, _ = make(dev, lens, T, H, 16, 51)
    g = torch.Generator().manual_seed(52)
    x = small * (1 + torch.rand(q.shape, generator=g))
    x[..., 0:512:8] = 64.0
    x[..., 512:] = 0.0
    q.copy_(x.bfloat16())
    codes = cache[..., :256].cpu() & 0x77                                       # all positive
    codes[..., 0:256:8] = codes[..., 0:256:8] & 0xf0 | 0x07
    codes[..., 4:256:8] = codes[..., 4:256:8] & 0xf0 | 0x0f
    cache[..., :256] = codes.to(dev)
    used = (cache[..., 256:272] != 255).all(-1, keepdim=True)
    cache[..., 256:272] = torch.where(used, 127, 255).to(torch.uint8)
    scale = 0.5
    o, lse = rda.rda_mla_decode_q4(q, cache, table, kl, scale, want_lse=True)
    for b, n in enumerate(lens):
        k = ref.cached(cache.cpu(), table[b].cpu(), n)
        for t in range(T):
            keys = k[:n - (T - 1 - t)]
            y = q[b, t].cpu().double()
            s = scale * (y @ keys.T)
            want = torch.logsumexp(s, 1)
            p = torch.exp(s - want[:, None])
            # two chains of 64 sums of eight, 4 instructions and 32 shared channels each, in 24
            # bits; and what the small channels lose
            small_ones = (y.abs() < 1)[:, :LATENT].double()
            lost = 32 * (2.0 ** -15 * small_ones @ keys[:, :LATENT].abs().T + 2.0 ** -14 * small_ones.sum(1, keepdim=True))
            ds = scale * (200 * 2.0 ** -23 * y.abs() @ keys.abs().T + lost).amax(1)
            c, h = keys.shape[0], BF16_HALF_STEP
            ro, most = p @ keys[:, :LATENT], p @ keys[:, :LATENT].abs()
            bo = h * ro.abs() + (h * (1 + h) + 2 * torch.expm1(ds)[:, None] + c * 2.0 ** -23) * most + 1e-38
            ref.check("o", o[b, t], ro, bo)
            ref.check("lse", lse[b, t], want, ds + (c + 16) * 2.0 ** -23 + 2.0 ** -22 * want.abs())
