"""GPU tests that the latent-attention and verification entry points write
their outputs and nothing beside them, every element of them, and that a
workspace's former contents (infinities and NaN included) do not matter."""
import pytest
import torch

from gated_delta_amd import rda
from gpu_util import guarded, need_gpu, say
from test_gpu_mla_decode import SCALE, make
from test_gpu_mla_prefill_wide import make as make_prompt, offsets
from test_gpu_verify import make as make_drafts

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.mark.parametrize("lens,T,H,prefix", [
    ([777], 1, 32, 0), ([777, 0, 5], 3, 40, 0), ([257, 900], 1, 4, 0), ([300, 2, 0], 2, 30, 0),
    ([100] * 40, 3, 32, 0), ([70, 0], 1, 32, 700), ([1, 0, 64], 5, 24, 33), ([20] * 60, 4, 33, 130),
])
def test_decode(dev, lens, T, H, prefix):
    say(f"[mla memory] decode lens={len(lens)} T={T} H={H} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, 16, 3, prefix)
    kw = dict(prefix_table=pre, prefix_len=prefix)
    want = rda.rda_mla_decode(q, cache, table, kl, SCALE, want_lse=True, **kw)
    B = len(lens)
    need = rda.rda_mla_decode_workspace_bytes(B, T, H, prefix)
    for byte in (0x00, 0xFF, 0x7F, 0x80):     # zeros, NaN, huge values, tiny negative ones
        o, lse = guarded((B, T, H, 512), BF16, dev), guarded((B, T, H), F32, dev)
        ws = guarded((need,), torch.uint8, dev)
        ws.t.fill_(byte)
        rda.rda_mla_decode(q, cache, table, kl, SCALE, o=o.t, lse=lse.t, workspace=ws.t, **kw)
        torch.cuda.synchronize()
        assert torch.equal(o.t, want[0]) and torch.equal(lse.t, want[1]), hex(byte)
        for x, name in ((o, "o"), (lse, "lse"), (ws, "workspace")):
            x.check(name)


@pytest.mark.parametrize("lq,lk,H", [
    ([1], [1], 3), ([33, 0, 130], [40, 5, 130], 4), ([400, 300], [400, 500], 80), ([2300, 1], [2300, 2100], 64),
])
def test_prefill(dev, lq, lk, H):
    say(f"[mla memory] prefill lq={lq} H={H}")
    q, kv, pe = make_prompt(dev, lq, lk, H, 4)
    want = rda.rda_mla_prefill(q, kv, pe, SCALE, offsets(lq), offsets(lk), want_lse=True)
    o, lse = guarded((sum(lq), H, 128), BF16, dev), guarded((sum(lq), H), F32, dev)
    rda.rda_mla_prefill(q, kv, pe, SCALE, offsets(lq), offsets(lk), o=o.t, lse=lse.t)
    torch.cuda.synchronize()
    assert torch.equal(o.t, want[0]) and torch.equal(lse.t, want[1])
    o.check("o")
    lse.check("lse")


@pytest.mark.parametrize("lq,H", [([3, 60], 4), ([200, 100], 40)])
def test_prompt_rows_behind_the_last_sequence_stay(dev, lq, H):
    """A packed batch padded behind its last sequence: those rows are left."""
    say(f"[mla memory] padded prompts lq={lq} H={H}")
    pad = 77
    q, kv, pe = make_prompt(dev, lq + [pad], lq + [pad], H, 5)
    cu = torch.tensor(offsets(lq), dtype=I32, device=dev)
    n = sum(lq)
    o = torch.full((n + pad, H, 128), 3.0, dtype=BF16, device=dev)
    lse = torch.full((n + pad, H), 5.0, device=dev)
    rda.rda_mla_prefill(q, kv, pe, SCALE, cu, o=o, lse=lse)
    want = rda.rda_mla_prefill(q[:n], kv[:n], pe[:n], SCALE, cu, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(o[:n], want[0]) and torch.equal(lse[:n], want[1])
    assert bool((o[n:] == 3).all()) and bool((lse[n:] == 5).all())


def test_append_padded(dev):
    """Rows of a packed batch behind its last sequence are not written."""
    _, cache, table, kl, _ = make(dev, [20, 9], 1, 1, 8, 6)
    cache = cache.nan_to_num(0.5)
    rows = torch.randn(40, 576, device=dev).bfloat16()
    cu = torch.tensor([0, 3, 7], dtype=I32, device=dev)
    g = guarded(tuple(cache.shape), BF16, dev)
    g.t.copy_(cache)
    rda.rda_mla_append(rows, g.t, table, kl, cu)
    want = rda.rda_mla_append(rows[:7], cache.clone(), table, kl, cu)
    torch.cuda.synchronize()
    assert torch.equal(g.t, want) and int((want != cache).any(-1).sum()) == 7
    g.check("cache")


@pytest.mark.parametrize("V,D,sampled", [(1, 0, True), (4097, 3, True), (30000, 7, False), (300001, 2, True)])
def test_verify(dev, V, D, sampled):
    say(f"[mla memory] verify V={V} D={D}")
    target, draft, tok, u, num = (None if x is None else x.to(dev) for x in make_drafts(5, D, V, V, sampled, True))
    want = rda.rda_verify_drafts(target, draft, tok, u, num)
    for byte in (0x00, 0xFF, 0x7F, 0x80):
        acc, out = guarded((5,), I32, dev), guarded((5, D + 1), I32, dev)
        ws = guarded((rda.rda_verify_drafts_workspace_bytes(5, V),), torch.uint8, dev)
        ws.t.fill_(byte)
        rda.rda_verify_drafts(target, draft, tok, u, num, accept=acc.t, out_tokens=out.t, workspace=ws.t)
        torch.cuda.synchronize()
        assert torch.equal(acc.t, want[0]) and torch.equal(out.t, want[1]), hex(byte)
        for x, name in ((acc, "accept"), (out, "out_tokens"), (ws, "workspace")):
            x.check(name)
