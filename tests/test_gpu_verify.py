"""GPU tests of rda_verify_drafts against the plain 64-bit form: the counts
and tokens are equal, not near."""
import pytest
import torch

import mla_ref
from gated_delta_amd import rda
from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def make(B, D, V, seed, sampled=True, ragged=False, sharp=2.0, noise=0.7):
    g = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(B, D + 1, V, generator=g)
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :D] + noise * torch.randn(B, D, V, generator=g), -1)
    if D:
        tok = (torch.multinomial(draft.reshape(B * D, V), 1, generator=g).reshape(B, D) if sampled
               else draft.argmax(-1))
    else:
        tok = torch.zeros(B, 0)
    u = torch.rand(B, D + 1, generator=g)
    num = torch.randint(0, D + 1, (B,), generator=g).to(torch.int32) if ragged else None
    return target, draft if sampled else None, tok.to(torch.int32), u, num


def run(dev, target, draft, tok, u, num=None):
    want = mla_ref.verify(target, draft, tok, u, num)
    up = lambda x: None if x is None else x.to(dev)
    acc, out = rda.rda_verify_drafts(up(target), up(draft), up(tok), up(u), up(num))
    torch.cuda.synchronize()
    assert acc.tolist() == want[0]
    assert out.tolist() == want[1]
    return acc, out


@pytest.mark.parametrize("V", [1, 2, 3, 64, 255, 256, 1009, 4095, 4096, 4097, 32003, 40000])
@pytest.mark.parametrize("sampled", [True, False])
def test_vocabularies(dev, V, sampled):
    say(f"[verify] V={V} sampled={sampled}")
    run(dev, *make(6, 2, V, V, sampled))


@pytest.mark.parametrize("D", [0, 1, 3, 7, 63])
@pytest.mark.parametrize("ragged", [True, False])
def test_draft_counts(dev, D, ragged):
    say(f"[verify] D={D} ragged={ragged}")
    run(dev, *make(9, D, 500, D, True, ragged, noise=0.1))


def test_whole_vocabulary(dev):
    """The models' vocabulary; more chunks than one scan of a workgroup never
    occur below a million tokens, so that too."""
    run(dev, *make(2, 1, 259840, 1, sharp=3.0))
    run(dev, *make(1, 1, 1200001, 2, sharp=1.0))


def test_borders(dev):
    """Random numbers at the borders of exactly representable sums: the
    smallest token whose running sum is greater."""
    p = torch.tensor([0.25, 0.0, 0.25, 0.5]).repeat(6, 1, 1).reshape(6, 1, 4)
    u = torch.tensor([0.0, 0.25, 0.49999997, 0.5, 0.99999994, 1.0]).reshape(6, 1)
    _, out = run(dev, p, None, torch.zeros(6, 0, dtype=torch.int32), u)
    assert out.flatten().tolist() == [0, 2, 2, 3, 3, 3]


def test_equal_rows_are_accepted(dev):
    """p = q: every draft stands; u q < p is strict, so u = 1 refuses and what
    is left of the target is nothing: then the target's own probabilities."""
    target, draft, tok, u, _ = make(4, 2, 100, 3, noise=0.0)
    acc, _ = run(dev, target, draft, tok, u)
    assert acc.tolist() == [3] * 4
    u = torch.ones_like(u)
    acc, _ = run(dev, target, target[:, :2].clone(), tok, u)
    assert acc.tolist() == [1] * 4


def test_nothing_weighs(dev):
    target, draft, tok, u, _ = make(3, 1, 70, 4)
    target[1] = 0
    target[2] = float("nan")
    _, out = run(dev, target, draft, tok, u)
    assert out[1, 0] == -1 and out[2, 0] == -1


def test_bad_values_weigh_nothing(dev):
    target, draft, tok, u, _ = make(4, 1, 5000, 5)
    target[:, :, 17] = float("nan")
    target[:, :, 4500] = float("inf")
    target[:, :, 30] = -1
    run(dev, target, draft, tok, u)


def test_tokens_out_of_range_are_refused(dev):
    target, draft, tok, u, _ = make(3, 3, 50, 6, noise=0.0)
    tok[0, 1], tok[1, 0], tok[2, 2] = -1, 50, 1 << 30
    acc, _ = run(dev, target, draft, tok, u * 0.5)
    assert acc.tolist() == [2, 1, 3]
    run(dev, target, None, tok, u)


def test_num_drafts_is_clamped(dev):
    target, draft, tok, u, _ = make(2, 2, 50, 7, noise=0.0)
    acc, _ = run(dev, target, draft, tok, u * 0.5, torch.tensor([-4, 99], dtype=torch.int32))
    assert acc.tolist() == [1, 3]


def test_row_strides(dev):
    target, draft, tok, u, _ = make(3, 2, 1001, 8)
    wide = torch.full((3, 3, 1024), 9.0)
    wide[..., :1001] = target
    wd = torch.full((3, 2, 1005), 9.0)
    wd[..., :1001] = draft
    want = mla_ref.verify(target, draft, tok, u)
    acc, out = rda.rda_verify_drafts(wide.to(dev)[..., :1001], wd.to(dev)[..., :1001], tok.to(dev), u.to(dev))
    assert (acc.tolist(), out.tolist()) == want


def test_distribution(dev):
    """Accepted or drawn again, the first token follows the target's
    distribution: frequencies over 60000 sequences against p, within five
    standard deviations."""
    B, V = 60000, 8
    g = torch.Generator().manual_seed(9)
    p = torch.softmax(torch.randn(V, generator=g), 0)
    q = torch.softmax(torch.randn(V, generator=g), 0)
    tok = torch.multinomial(q, B, replacement=True, generator=g).to(torch.int32).reshape(B, 1)
    u = torch.rand(B, 2, generator=g)
    target = p.expand(B, 2, V).contiguous().to(dev)
    draft = q.expand(B, 1, V).contiguous().to(dev)
    _, out = rda.rda_verify_drafts(target, draft, tok.to(dev), u.to(dev))
    freq = torch.bincount(out[:, 0].cpu().long(), minlength=V).double() / B
    dev5 = 5 * torch.sqrt(p.double() * (1 - p.double()) / B)
    assert bool(((freq - p.double()).abs() < dev5).all())


def test_graph_replays(dev):
    target, draft, tok, u, _ = (None if x is None else x.to(dev) for x in make(5, 2, 3001, 10))
    acc, out = rda.rda_verify_drafts(target, draft, tok, u)
    ws = torch.empty(rda.rda_verify_drafts_workspace_bytes(5, 3001), dtype=torch.uint8, device=dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rda.rda_verify_drafts(target, draft, tok, u, accept=acc, out_tokens=out, workspace=ws)
    for seed in range(3):
        u.copy_(torch.rand(5, 3, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        want = mla_ref.verify(target.cpu(), draft.cpu(), tok.cpu(), u.cpu())
        assert (acc.tolist(), out.tolist()) == want
