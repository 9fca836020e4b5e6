"""GPU tests of rda_mla_decode_q4 (absorbed latent attention over the 4-bit
cache, with and without a shared prefix) against the 64-bit form."""
import pytest
import torch

import mla_q4_ref as ref
from gated_delta_amd import rda
from gpu_util import guarded, need_gpu, say

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def random_rows(n, g, exponents=(-2, 2)):
    """Rows of random codes, scales 2^exponents and normal shared channels."""
    rows = torch.randint(0, 256, (n, 400), generator=g, dtype=torch.int32).to(torch.uint8)
    rows[:, 256:272] = torch.randint(127 + exponents[0], 128 + exponents[1], (n, 16), generator=g).to(torch.uint8)
    rows[:, 272:] = torch.randn(n, 64, generator=g).bfloat16().view(torch.uint8)
    return rows


def make(dev, lens, T, H, page, seed, prefix=0, spread=0.3, spare=2, width=None):
    """Queries, a shuffled page pool whose unused rows are NaN, tables."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    npre = -(-prefix // page)
    pool = sum(need) + npre + spare
    cache = torch.full((pool, page, 400), 255, dtype=torch.uint8)   # scales and shared channels: NaN
    perm = torch.randperm(pool, generator=g).tolist()
    width = width or max(1, max(need, default=1))
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0

    def fill(n):
        nonlocal at
        pages = perm[at:at + -(-n // page)]
        at += len(pages)
        rows = random_rows(n, g)
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


def compare(q, cache, table, kl, pre, prefix, lens):
    dev = q.device
    B, T, H, _ = q.shape
    go, gl = guarded((B, T, H, 512), torch.bfloat16, dev), guarded((B, T, H), torch.float32, dev)
    o, lse = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=prefix,
                                   o=go.t, lse=gl.t)
    torch.cuda.synchronize()
    go.check("o")
    gl.check("lse")
    ro, rl, bo, bl = ref.decode(q, cache, table.cpu(), lens, SCALE, None if pre is None else pre.cpu(), prefix)
    ref.check("o", o, ro, bo)
    ref.check("lse", lse, rl, bl)
    return o, lse


def run(dev, lens, T, H, page, seed=0, prefix=0, spread=0.3):
    say(f"[mla decode q4] lens={lens if len(lens) < 12 else len(lens)} T={T} H={H} page={page} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, page, seed, prefix, spread)
    return compare(q, cache, table, kl, pre, prefix, lens)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 33, 63, 64, 65, 127, 128, 129, 300, 1100])
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
    run(dev, [1, 63, 64, 200, 7], 2, 8, page, seed=page)


def test_empty_and_short(dev):
    """No rows, fewer rows than new tokens: those tokens get 0 and -inf."""
    o, lse = run(dev, [0, 1, 2, 3, 70], 4, 5, 16, seed=3)
    assert float(o[0].float().abs().max()) == 0 and bool(torch.isinf(lse[0]).all())


@pytest.mark.parametrize("lens,T,H", [([3000], 1, 32), ([3000, 1, 0, 2500], 3, 16), ([900] * 9, 3, 32),
                                      ([5] * 300, 1, 8), (list(range(0, 520, 2)), 1, 4)])
def test_split_and_shared_work(dev, lens, T, H):
    run(dev, lens, T, H, 64, seed=len(lens))


@pytest.mark.parametrize("lens,T,H,prefix", [([0, 3, 50], 1, 8, 1), ([5, 0, 64], 2, 40, 65),
                                             ([1] * 8, 1, 32, 1000), ([30] * 70, 3, 32, 300),
                                             ([0] * 5, 1, 4, 130)])
def test_prefix(dev, lens, T, H, prefix):
    run(dev, lens, T, H, 64, seed=prefix, prefix=prefix)


@pytest.mark.parametrize("spread", [0.0, 3.0, 30.0])
def test_score_ranges(dev, spread):
    """All scores alike; a softmax with one large term, whose maximum comes late or early."""
    run(dev, [400, 257], 2, 6, 32, seed=11, spread=spread)
