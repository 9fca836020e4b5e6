"""GPU tests of rda_verify_drafts at values that its own bookkeeping or its
differences could take for something else, with answers worked out by hand."""
import pytest
import torch

from gated_delta_amd import rda
from gpu_util import need_gpu, say
from test_gpu_verify import make, run

pytestmark = pytest.mark.gpu
INT_MIN = -(1 << 31)


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.mark.parametrize("token", [INT_MIN, INT_MIN + 1, -1, 2, (1 << 31) - 1])
def test_any_token_out_of_range_is_a_refusal(dev, token):
    """p = (1/2, 1/2), q = (1, 0): what is left after the refusal is (0, 1/2)."""
    say(f"[verify] refused token {token}")
    p = torch.tensor([0.5, 0.5]).repeat(1, 2, 1).to(dev)
    q = torch.tensor([[[1.0, 0.0]]], device=dev)
    tok = torch.tensor([[token]], dtype=torch.int32, device=dev)
    acc, out = rda.rda_verify_drafts(p, q, tok, torch.tensor([[0.0, 0.1]], device=dev))
    assert acc.tolist() == [1] and out.tolist() == [[1, -1]]
    # without draft probabilities nothing is taken from the target's
    acc, out = rda.rda_verify_drafts(p, None, tok, torch.tensor([[0.0, 0.1]], device=dev))
    assert acc.tolist() == [1] and out.tolist() == [[0, -1]]


@pytest.mark.parametrize("V", [50, 9001])
def test_smallest_token_among_others(dev, V):
    target, draft, tok, u, num = make(8, 3, V, V, noise=1.0)
    tok[::2, 1] = INT_MIN
    run(dev, target, draft, tok, u, num)
    run(dev, target, None, tok, u, num)


@pytest.mark.parametrize("p0", [-1.0, 0.0, float("nan"), float("-inf"), float("inf")])
@pytest.mark.parametrize("q0", [-2.0, float("-inf"), 0.0])
def test_a_target_that_is_not_positive_and_finite_weighs_nothing(dev, p0, q0):
    """Whatever the draft row holds there: p = (p0, 1/2, 1/2), q = (q0, 0, 1/4)
    leave (0, 1/2, 1/4)."""
    p = torch.tensor([p0, 0.5, 0.5]).repeat(4, 2, 1).to(dev)
    q = torch.tensor([q0, 0.0, 0.25]).repeat(4, 1, 1).to(dev)
    u = torch.tensor([[0.0, 0.0], [0.0, 0.6], [0.0, 0.7], [0.0, 0.99]], device=dev)
    tok = torch.full((4, 1), -1, dtype=torch.int32, device=dev)
    acc, out = rda.rda_verify_drafts(p, q, tok, u)
    assert acc.tolist() == [1] * 4 and out[:, 0].tolist() == [1, 1, 2, 2]
