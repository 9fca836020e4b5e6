"""GPU tests of calls on two streams at once that make their own memory: a
call on the current stream is followed by one on another, nothing waits
between them, and what either leaves behind at once goes to the next."""
import pytest
import torch

from gated_delta_amd import rda
from gpu_util import need_gpu, say
from test_gpu_mla_decode import SCALE, make
from test_gpu_verify import make as make_drafts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def alternate(fn, want, same):
    """fn(None) and fn(side stream) in turn, without a wait; all like `want`."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [fn(s) for _ in range(6) for s in (None, side)]
    torch.cuda.synchronize()
    for i, x in enumerate(outs):
        assert same(x, want), f"call {i}"


def equal(a, b):
    return all(x is None and y is None or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("prefix", [0, 500])
def test_decode(dev, prefix):
    """Two batches of other lengths, so that a workspace shared by mistake
    would hold other plans."""
    say(f"[mla streams] decode prefix={prefix}")
    args = [make(dev, lens, 1, 32, 64, 3, prefix) for lens in ([700, 300, 2000], [1500, 1, 40])]

    def fn(s, which):
        q, cache, table, kl, pre = args[which]
        return rda.rda_mla_decode(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=prefix,
                                  want_lse=True, stream=s)

    want = [fn(None, 0), fn(None, 1)]
    alternate(lambda s: fn(s, 0) + fn(s, 1), want[0] + want[1], equal)


def test_prefill_and_append_with_lists(dev):
    say("[mla streams] prefill and append, offsets as lists")
    g = torch.Generator().manual_seed(4)
    lens = [50, 200, 1, 149]
    cu = [0, 50, 250, 251, 400]
    q = torch.randn(400, 4, 192, generator=g).bfloat16().to(dev)
    kv = torch.randn(400, 4, 256, generator=g).bfloat16().to(dev)
    rows = torch.randn(400, 576, generator=g).bfloat16().to(dev)
    table = torch.randperm(32, generator=g).to(torch.int32).reshape(4, 8).to(dev)
    kl = torch.tensor(lens, dtype=torch.int32, device=dev)
    caches = [torch.zeros(32, 32, 576, dtype=torch.bfloat16, device=dev) for _ in range(13)]
    at = iter(caches)

    def fn(s):
        c = rda.rda_mla_append(rows, next(at), table, kl, cu, stream=s)
        o, lse = rda.rda_mla_prefill(q, kv, rows[:, 512:], SCALE, cu, want_lse=True, stream=s)
        filler = torch.full((5,), 7, dtype=torch.int32, device=dev)   # what a lost temporary would become
        return c, o, lse, filler

    alternate(fn, fn(None), equal)


def test_verify(dev):
    say("[mla streams] verify")
    args = [[None if x is None else x.to(dev) for x in make_drafts(9, 3, 20011, seed)] for seed in (1, 2)]
    want = [rda.rda_verify_drafts(*a) for a in args]
    alternate(lambda s: rda.rda_verify_drafts(*args[0], stream=s) + rda.rda_verify_drafts(*args[1], stream=s),
              want[0] + want[1], equal)


def test_outputs_let_go_at_once(dev):
    """Outputs that are dropped while their call still runs, between calls on
    the current stream that allocate as much."""
    say("[mla streams] dropped outputs")
    q, cache, table, kl, _ = make(dev, [3000, 500], 1, 32, 64, 5)
    want, _ = rda.rda_mla_decode(q, cache, table, kl, SCALE)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        rda.rda_mla_decode(q, cache, table, kl, SCALE, stream=side)
        kept = torch.full_like(want, 3)
        got, _ = rda.rda_mla_decode(q, cache, table, kl, SCALE)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and bool((kept == 3).all())
