"""GPU tests of the serving entry points together: a prompt's latent rows go to
the cache and its queries through rda_mla_prefill; then steps of a current token
and its drafts through rda_mla_append, rda_mla_decode, rda_verify_drafts and
rda_decode_tokens, eagerly and as one captured graph.  Also rda_mla_decode at
batches whose sequences are shared out in different ways."""
import pytest
import torch

import mla_ref
from gated_delta_amd import rda
from gpu_util import need_gpu, say
from test_gpu_mla_decode import bound_append, run as decode_run

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


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
    ([0, 0, 700, 0, 33, 1] * 8, 3, 24),    # empty ones between, blocks of 128 rows
    (spread(250, 1, 40, 4), 1, 8),         # nearly as many sequences as workgroups
    (spread(250, 40, 300, 4), 1, 4),       # more shares than workgroups: equal shares
    (spread(300, 0, 90, 5), 1, 4),         # more sequences than workgroups
    ([5000] + [1] * 30, 1, 8),             # one long, many short
    (spread(40, 1, 200, 6), 5, 32),        # two blocks of 128 rows a sequence
])
def test_shares(dev, lens, T, H):
    decode_run(dev, lens, T, H, 32, seed=len(lens) + T)


@pytest.mark.parametrize("lens,T,H,prefix", [
    ([17, 33, 0, 1] * 6, 1, 40, 11),       # a prefix of less than a tile, many blocks
    ([5, 2] * 9, 3, 16, 70),
    (spread(20, 0, 60, 7), 8, 120, 40),    # many rows of a short prefix
])
def test_short_prefixes(dev, lens, T, H, prefix):
    decode_run(dev, lens, T, H, 16, seed=len(lens) + T, prefix=prefix)


def test_prompt_then_tokens(dev):
    """Prompts of several lengths: rows into the cache, keys and values from the
    cached rows, the prompt's attention; then one more token by the absorbed form."""
    lens, H, page = [70, 1, 200, 33], 4, 32
    g = torch.Generator().manual_seed(1)
    rows = torch.randn(sum(lens), 576, generator=g).bfloat16()
    weight = 1 + 0.1 * torch.randn(512, generator=g)
    wk = torch.randn(H, 128, 512, generator=g) * 512 ** -0.5
    wv = torch.randn(H, 128, 512, generator=g) * 512 ** -0.5
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    width = 8
    table = torch.randperm(len(lens) * width, generator=g).to(torch.int32).reshape(len(lens), width)
    cache = torch.zeros(len(lens) * width, page, 576, dtype=torch.bfloat16)
    say(f"[mla serving] prompts {lens}, then one token each")
    d = {n: t.to(dev) for n, t in dict(rows=rows, weight=weight, table=table, cache=cache).items()}
    kl = torch.tensor(lens, dtype=torch.int32, device=dev)
    cud = torch.tensor(cu, dtype=torch.int32, device=dev)
    rda.rda_mla_append(d["rows"], d["cache"], d["table"], kl, cud, weight=d["weight"])
    torch.cuda.synchronize()
    ref = mla_ref.append(rows, cache, table, lens, cu, weight, 1e-5)
    mla_ref.check("cache", d["cache"], ref, bound_append(ref))
    cached = torch.cat([mla_ref.cached_rows(d["cache"].cpu(), table[b], n) for b, n in enumerate(lens)])
    c = cached[:, :512].double()
    kv = torch.stack([torch.cat([c @ wk[h].double().T, c @ wv[h].double().T], 1) for h in range(H)], 1).bfloat16()
    q = torch.randn(sum(lens), H, 192, generator=g).bfloat16()
    o, lse = rda.rda_mla_prefill(q.to(dev), kv.to(dev), cached.to(dev)[:, 512:], SCALE, cud, want_lse=True)
    torch.cuda.synchronize()
    ro, rl, bo, bl = mla_ref.prefill(q, kv, cached[:, 512:], SCALE, cu, cu, True)
    mla_ref.check("prompt o", o, ro, bo)
    mla_ref.check("prompt lse", lse, rl, bl)
    # the next token
    one = torch.randn(len(lens), 576, generator=g).bfloat16()
    kl += 1
    rda.rda_mla_append(one.to(dev), d["cache"], d["table"], kl, weight=d["weight"])
    qn = torch.randn(len(lens), H, 192, generator=g)
    qa = torch.cat([torch.einsum("bhd,hdc->bhc", qn[..., :128], wk), qn[..., 128:]], -1).bfloat16()[:, None].contiguous()
    o, lse = rda.rda_mla_decode(qa.to(dev), d["cache"], d["table"], kl, SCALE, want_lse=True)
    torch.cuda.synchronize()
    ro, rl, bo, bl = mla_ref.decode(qa, d["cache"].cpu(), table, kl.tolist(), SCALE)
    mla_ref.check("token o", o, ro, bo)
    mla_ref.check("token lse", lse, rl, bl)


class Steps:
    """B sequences that take a current token and D drafts per step, in fixed buffers."""

    def __init__(self, dev, B=5, D=3, H=4, V=1009, page=16):
        self.dev, self.B, self.T, self.H, self.V = dev, B, D + 1, H, V
        g = torch.Generator().manual_seed(3)
        width = 12
        self.table = torch.randperm(B * width, generator=g).to(torch.int32).reshape(B, width).to(dev)
        self.cache = torch.randn(B * width, page, 576, generator=g).bfloat16().to(dev)
        self.committed = torch.tensor([0, 1, 40, 16, 63][:B], dtype=torch.int32, device=dev)
        self.weight = (1 + 0.1 * torch.randn(512, generator=g)).to(dev)
        self.S = (0.1 * torch.randn(B, H, 128, 128, generator=g)).to(dev)
        self.lens, self.accept = torch.empty_like(self.committed), torch.empty_like(self.committed)
        self.tokens = torch.empty(B, self.T, dtype=torch.int32, device=dev)
        self.o = torch.empty(B, self.T, H, 512, dtype=torch.bfloat16, device=dev)
        self.mix = torch.empty(B, self.T, H, 128, device=dev)
        self.ws = torch.empty(rda.rda_mla_decode_workspace_bytes(B, self.T, H, 0), dtype=torch.uint8, device=dev)
        self.wv = torch.empty(rda.rda_verify_drafts_workspace_bytes(B, V), dtype=torch.uint8, device=dev)
        self.load(0)

    def load(self, n):
        g = torch.Generator().manual_seed(50 + n)
        B, T, H, V = self.B, self.T, self.H, self.V

        def put(name, t):
            if hasattr(self, name):
                getattr(self, name).copy_(t)
            else:
                setattr(self, name, t.to(self.dev))

        put("rows", torch.randn(B * T, 576, generator=g).bfloat16())
        put("q", torch.randn(B, T, H, 576, generator=g).bfloat16())
        logits = 2 * torch.randn(B, T, V, generator=g)
        near = logits[:, :-1] + 0.3 * torch.randn(B, T - 1, V, generator=g)
        put("target", torch.softmax(logits, -1))
        draft = torch.softmax(near, -1)
        put("draft", draft)
        put("drafted", torch.multinomial(draft.reshape(-1, V), 1, generator=g).reshape(B, T - 1).to(torch.int32))
        put("u", torch.rand(B, T, generator=g))
        for name in ("mq", "mk", "mv"):
            put(name, torch.nn.functional.normalize(torch.randn(B, T, H, 128, generator=g), dim=-1).bfloat16())
        put("a", -torch.rand(B, T, H, generator=g))
        put("b", torch.rand(B, T, H, generator=g))

    def step(self):
        torch.add(self.committed, self.T, out=self.lens)
        rda.rda_mla_append(self.rows, self.cache, self.table, self.lens, weight=self.weight)
        rda.rda_mla_decode(self.q, self.cache, self.table, self.lens, SCALE, o=self.o, workspace=self.ws)
        rda.rda_verify_drafts(self.target, self.draft, self.drafted, self.u, accept=self.accept,
                              out_tokens=self.tokens, workspace=self.wv)
        rda.rda_decode_tokens(self.mq, self.mk, self.mv, self.a, self.b, self.S, S_out=self.S,
                              accept=self.accept, o=self.mix)
        self.committed.add_(self.accept)


def test_speculative_steps(dev):
    """Three steps: each one's attention sees the rows kept so far and its own,
    verification says how many stay, the mixer's state takes as many tokens."""
    s = Steps(dev)
    for n in range(3):
        s.load(n)
        kept, S0 = s.committed.tolist(), s.S.clone()
        before = s.cache.cpu()
        s.step()
        torch.cuda.synchronize()
        say(f"[mla serving] step {n}: kept {kept}, accepted {s.accept.tolist()}")
        lens = [k + s.T for k in kept]
        cu = [s.T * i for i in range(s.B + 1)]
        ref = mla_ref.append(s.rows, before, s.table.cpu(), lens, cu, s.weight, 1e-5)
        mla_ref.check("cache", s.cache, ref, bound_append(ref))
        ro, _, bo, _ = mla_ref.decode(s.q.cpu(), s.cache.cpu(), s.table.cpu(), lens, SCALE)
        mla_ref.check("o", s.o, ro, bo)
        acc, out = mla_ref.verify(s.target.cpu(), s.draft.cpu(), s.drafted.cpu(), s.u.cpu())
        assert s.accept.tolist() == list(acc) and s.tokens.tolist() == [list(x) for x in out]
        assert s.committed.tolist() == [k + a for k, a in zip(kept, acc)]
        # the state after as many tokens, one sequence and its own count at a time
        for b, a in enumerate(acc):
            one = torch.empty_like(S0[b:b + 1])
            part = [x[b:b + 1, :a].contiguous() for x in (s.mq, s.mk, s.mv, s.a, s.b)]
            rda.rda_decode_tokens(*part, S0[b:b + 1].contiguous(), S_out=one)
            assert torch.equal(one[0], s.S[b])


def test_speculative_steps_captured(dev):
    """The whole step as one graph, replayed between eager work of its own kind."""
    eager, graphed = Steps(dev), Steps(dev)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        Steps(dev).step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            graphed.step()
    torch.cuda.synchronize()
    for n in range(4):
        eager.load(n)
        graphed.load(n)
        graph.replay()
        torch.cuda.synchronize()
        eager.step()
        torch.cuda.synchronize()
        for name in ("cache", "o", "accept", "tokens", "mix", "S", "committed"):
            assert torch.equal(getattr(eager, name), getattr(graphed, name)), (n, name)
