"""GPU tests of the 4-bit latent cache as a server uses it: prompts in pieces,
then steps of a current token and its drafts, eagerly and as one captured graph;
calls on two streams; workspaces of any contents; nothing written beside the
outputs."""
import pytest
import torch

import mla_q4_ref as ref
import mla_ref
from gated_delta_amd import rda
from gpu_util import guarded, need_gpu, say
from test_gpu_mla_decode_q4 import SCALE, make
from test_gpu_mla_streams import alternate, equal

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def test_prompt_in_pieces_then_tokens(dev):
    """Prompts that come in two pieces: rows into the cache, all rows so far out of it
    again, keys and values up-projected from those, the piece's attention; then one
    more token by the absorbed form, which is also rda_mla_decode's over the rows that
    the cache stands for."""
    first, second, H, page = [70, 1, 0, 33], [30, 200, 17, 1], 4, 32
    N, width = len(first), 8
    g = torch.Generator().manual_seed(1)
    weight = (1 + 0.1 * torch.randn(512, generator=g)).to(dev)
    wk = torch.randn(H, 128, 512, generator=g) * 512 ** -0.5
    wv = torch.randn(H, 128, 512, generator=g) * 512 ** -0.5
    table = torch.randperm(N * width, generator=g).to(I32).reshape(N, width)
    td = table.to(dev)
    cache = torch.zeros(N * width, page, 400, dtype=torch.uint8, device=dev)

    def offsets(ns):
        out = [0]
        for n in ns:
            out.append(out[-1] + n)
        return out

    have = [0] * N
    for new in (first, second):
        say(f"[mla q4 serving] pieces {new} after {have}")
        have = [a + b for a, b in zip(have, new)]
        rows = torch.randn(sum(new), 576, generator=g).bfloat16()
        kl = torch.tensor(have, dtype=I32, device=dev)
        want = ref.append(rows, cache, table, have, offsets(new), weight, 1e-5)
        rda.rda_mla_append_q4(rows.to(dev), cache, td, kl, offsets(new), weight=weight)
        assert torch.equal(cache.cpu(), want)
        out = rda.rda_mla_read_q4(cache, td, kl, sum(have), offsets(have)).cpu()
        assert torch.equal(out.double(), ref.read(want, table, have, offsets(have), sum(have)))
        c = out[:, :512].double()
        kv = torch.stack([torch.cat([c @ wk[h].double().T, c @ wv[h].double().T], 1) for h in range(H)], 1).bfloat16()
        q = torch.randn(sum(new), H, 192, generator=g).bfloat16()
        o, lse = rda.rda_mla_prefill(q.to(dev), kv.to(dev), out.to(dev)[:, 512:], SCALE, offsets(new), offsets(have),
                                     want_lse=True)
        torch.cuda.synchronize()
        ro, rl, bo, bl = mla_ref.prefill(q, kv, out[:, 512:], SCALE, offsets(new), offsets(have), True)
        mla_ref.check("prompt o", o, ro, bo)
        mla_ref.check("prompt lse", lse, rl, bl)
    # the next token
    have = [n + 1 for n in have]
    kl += 1
    rda.rda_mla_append_q4(torch.randn(N, 576, generator=g).bfloat16().to(dev), cache, td, kl, weight=weight)
    qn = torch.randn(N, H, 192, generator=g)
    qa = torch.cat([torch.einsum("bhd,hdc->bhc", qn[..., :128], wk), qn[..., 128:]], -1).bfloat16()[:, None].contiguous().to(dev)
    o, lse = rda.rda_mla_decode_q4(qa, cache, td, kl, SCALE, want_lse=True)
    ro, rl, bo, bl = ref.decode(qa, cache, table, have, SCALE)
    ref.check("token o", o, ro, bo)
    ref.check("token lse", lse, rl, bl)
    plain = torch.zeros(N * width, page, 576, dtype=BF16, device=dev)
    rows = rda.rda_mla_read_q4(cache, td, kl, sum(have), offsets(have))
    rda.rda_mla_append(rows, plain, td, kl, offsets(have))
    po, pl = rda.rda_mla_decode(qa, plain, td, kl, SCALE, want_lse=True)
    ref.check("bf16 cache's o", po, ro, bo)
    ref.check("bf16 cache's lse", pl, rl, bl)


class Steps:
    """B sequences that take a current token and D drafts per step, in fixed buffers."""

    def __init__(self, dev, B=5, D=3, H=12, V=1009, page=16):
        self.dev, self.B, self.T, self.H, self.V = dev, B, D + 1, H, V
        g = torch.Generator().manual_seed(3)
        width = 12
        self.table = torch.randperm(B * width, generator=g).to(I32).reshape(B, width).to(dev)
        self.cache = torch.zeros(B * width, page, 400, dtype=torch.uint8, device=dev)
        self.committed = torch.tensor([0, 1, 40, 16, 63][:B], dtype=I32, device=dev)
        self.weight = (1 + 0.1 * torch.randn(512, generator=g)).to(dev)
        self.lens, self.accept = torch.empty_like(self.committed), torch.empty_like(self.committed)
        self.tokens = torch.empty(B, self.T, dtype=I32, device=dev)
        self.o = torch.empty(B, self.T, H, 512, dtype=BF16, device=dev)
        self.back = torch.empty(B * self.T, 576, dtype=BF16, device=dev)
        self.ws = torch.empty(rda.rda_mla_decode_q4_workspace_bytes(B, self.T, H, 0), dtype=torch.uint8, device=dev)
        self.wv = torch.empty(rda.rda_verify_drafts_workspace_bytes(B, V), dtype=torch.uint8, device=dev)
        have = int(self.committed.sum())
        cu = [0]
        for n in self.committed.tolist():
            cu.append(cu[-1] + n)
        rda.rda_mla_append_q4(torch.randn(have, 576, generator=g).bfloat16().to(dev), self.cache, self.table,
                              self.committed, cu, weight=self.weight)
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
        put("drafted", torch.multinomial(draft.reshape(-1, V), 1, generator=g).reshape(B, T - 1).to(I32))
        put("u", torch.rand(B, T, generator=g))

    def step(self):
        torch.add(self.committed, self.T, out=self.lens)
        rda.rda_mla_append_q4(self.rows, self.cache, self.table, self.lens, weight=self.weight)
        rda.rda_mla_decode_q4(self.q, self.cache, self.table, self.lens, SCALE, o=self.o, workspace=self.ws)
        rda.rda_mla_read_q4(self.cache, self.table, self.lens, self.B * self.T, out=self.back)
        rda.rda_verify_drafts(self.target, self.draft, self.drafted, self.u, accept=self.accept,
                              out_tokens=self.tokens, workspace=self.wv)
        self.committed.add_(self.accept)


def test_speculative_steps(dev):
    """Three steps: each one's attention sees the rows kept so far and its own; rows
    that were not kept are overwritten by the next."""
    s = Steps(dev)
    for n in range(3):
        s.load(n)
        kept, before = s.committed.tolist(), s.cache.cpu()
        s.step()
        torch.cuda.synchronize()
        say(f"[mla q4 serving] step {n}: kept {kept}, accepted {s.accept.tolist()}")
        lens, cu = [k + s.T for k in kept], [s.T * i for i in range(s.B + 1)]
        assert torch.equal(s.cache.cpu(), ref.append(s.rows, before, s.table.cpu(), lens, cu, s.weight, 1e-5))
        ro, _, bo, _ = ref.decode(s.q, s.cache, s.table.cpu(), lens, SCALE)
        ref.check("o", s.o, ro, bo)
        assert torch.equal(s.back.cpu().double(), ref.read(s.cache.cpu(), s.table.cpu(), lens, cu, s.B * s.T))
        assert s.committed.tolist() == [k + a for k, a in zip(kept, s.accept.tolist())]


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
        for name in ("cache", "o", "back", "accept", "tokens", "committed"):
            assert torch.equal(getattr(eager, name), getattr(graphed, name)), (n, name)


@pytest.mark.parametrize("prefix", [0, 300])
def test_captured_with_other_lengths(dev, prefix):
    """A captured call replayed with other lengths and tables: other plans."""
    say(f"[mla q4] captured, prefix={prefix}")
    B, H = 6, 16
    q, cache, table, kl, pre = make(dev, [500] * B, 1, H, 16, 12, prefix)
    o, lse = torch.empty(B, 1, H, 512, dtype=BF16, device=dev), torch.empty(B, 1, H, device=dev)
    ws = torch.empty(rda.rda_mla_decode_q4_workspace_bytes(B, 1, H, prefix), dtype=torch.uint8, device=dev)
    kw = dict(prefix_table=pre, prefix_len=prefix)
    call = lambda: rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, o=o, lse=lse, workspace=ws, **kw)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
    torch.cuda.synchronize()
    for lens in ([500] * B, [1, 0, 499, 33, 32, 31], [0] * B, [500, 1, 1, 1, 1, 1]):
        kl.copy_(torch.tensor(lens, dtype=I32))
        table.copy_(table.roll(1, 0))
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, want_lse=True, **kw)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), lens


@pytest.mark.parametrize("prefix", [0, 500])
def test_two_streams(dev, prefix):
    """Two batches of other lengths, so that a workspace shared by mistake would hold
    other plans."""
    say(f"[mla q4 streams] prefix={prefix}")
    args = [make(dev, lens, 1, 32, 64, 3, prefix) for lens in ([700, 300, 2000], [1500, 1, 40])]

    def fn(s, which):
        q, cache, table, kl, pre = args[which]
        out = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, prefix_table=pre, prefix_len=prefix, want_lse=True,
                                    stream=s)
        return *out, rda.rda_mla_read_q4(cache, table, kl, 50, [0, 40, 49, 50], stream=s)[:, :512].nan_to_num()

    want = [fn(None, 0), fn(None, 1)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        a, b = fn(None, 0)[:2], None
        o, lse = rda.rda_mla_decode_q4(*args[1][:4], SCALE, prefix_table=args[1][4], prefix_len=prefix, want_lse=True,
                                       stream=side)
        torch.cuda.synchronize()
        assert equal(a, want[0][:2]) and torch.equal(o, want[1][0]) and torch.equal(lse, want[1][1])


def test_append_and_read_with_lists_on_two_streams(dev):
    say("[mla q4 streams] append and read, offsets as lists")
    g = torch.Generator().manual_seed(4)
    cu = [0, 50, 250, 251, 400]
    rows = torch.randn(400, 576, generator=g).bfloat16().to(dev)
    table = torch.randperm(32, generator=g).to(I32).reshape(4, 8).to(dev)
    kl = torch.tensor([50, 200, 1, 149], dtype=I32, device=dev)
    caches = iter([torch.zeros(32, 32, 400, dtype=torch.uint8, device=dev) for _ in range(13)])

    def fn(s):
        c = rda.rda_mla_append_q4(rows, next(caches), table, kl, cu, stream=s)
        out = rda.rda_mla_read_q4(c, table, kl, 400, cu, stream=s)
        filler = torch.full((5,), 7, dtype=I32, device=dev)   # what a lost temporary would become
        return c, out, filler

    alternate(fn, fn(None), equal)


@pytest.mark.parametrize("lens,T,H,prefix", [
    ([777], 1, 32, 0), ([777, 0, 5], 3, 40, 0), ([257, 900], 1, 4, 0), ([300, 2, 0], 2, 30, 0),
    ([100] * 40, 3, 32, 0), ([70, 0], 1, 32, 700), ([1, 0, 64], 5, 24, 33), ([20] * 60, 4, 33, 130),
])
def test_memory(dev, lens, T, H, prefix):
    """Outputs and workspace are written within their bounds, and a workspace's former
    contents (infinities and NaN included) do not matter."""
    say(f"[mla q4 memory] lens={len(lens)} T={T} H={H} prefix={prefix}")
    q, cache, table, kl, pre = make(dev, lens, T, H, 16, 3, prefix)
    kw = dict(prefix_table=pre, prefix_len=prefix)
    want = rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, want_lse=True, **kw)
    B, kept = len(lens), cache.clone()
    need = rda.rda_mla_decode_q4_workspace_bytes(B, T, H, prefix)
    for byte in (0x00, 0xFF, 0x7F, 0x80):     # zeros, NaN, huge values, tiny negative ones
        o, lse = guarded((B, T, H, 512), BF16, dev), guarded((B, T, H), F32, dev)
        ws = guarded((need,), torch.uint8, dev)
        ws.t.fill_(byte)
        rda.rda_mla_decode_q4(q, cache, table, kl, SCALE, o=o.t, lse=lse.t, workspace=ws.t, **kw)
        torch.cuda.synchronize()
        assert torch.equal(o.t, want[0]) and torch.equal(lse.t, want[1]), hex(byte)
        for x, name in ((o, "o"), (lse, "lse"), (ws, "workspace")):
            x.check(name)
    assert torch.equal(cache, kept)


def test_padded_batches(dev):
    """Rows of a packed batch behind its last sequence: neither stored nor written."""
    say("[mla q4 memory] padded batches")
    _, cache, table, kl, _ = make(dev, [20, 9], 1, 1, 8, 6)
    rows = torch.randn(40, 576, device=dev).bfloat16()
    cu = torch.tensor([0, 3, 7], dtype=I32, device=dev)
    g = guarded(tuple(cache.shape), torch.uint8, dev)
    g.t.copy_(cache)
    rda.rda_mla_append_q4(rows, g.t, table, kl, cu)
    want = rda.rda_mla_append_q4(rows[:7], cache.clone(), table, kl, cu)
    torch.cuda.synchronize()
    assert torch.equal(g.t, want) and int((want != cache).any(-1).sum()) == 7
    g.check("cache")
    out = torch.full((40, 576), 3.0, dtype=BF16, device=dev)
    rda.rda_mla_read_q4(g.t, table, kl, 40, cu, out=out)
    assert torch.equal(out[:7], rda.rda_mla_read_q4(g.t, table, kl, 7, cu)) and bool((out[7:] == 3).all())


@pytest.mark.parametrize("total,seqs", [(8191, 1), (8192, 1), (9001, 3), (20000, 4000)])
def test_many_rows(dev, total, seqs):
    """Both forms of the reader (a wave reads one row, or two), and the writer, over
    many rows and sequences: what was written comes back."""
    say(f"[mla q4] {total} rows of {seqs} sequences")
    g = torch.Generator().manual_seed(total)
    cut = sorted(torch.randint(0, total + 1, (seqs - 1,), generator=g).tolist())
    cu = [0, *cut, total]
    lens = [b - a for a, b in zip(cu, cu[1:])]
    page = 16
    need = [-(-n // page) for n in lens]
    table = torch.full((seqs, max(need)), -1, dtype=I32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = torch.arange(at, at + n)
        at += n
    cache = torch.zeros(at, page, 400, dtype=torch.uint8, device=dev)
    table, kl = table.to(dev), torch.tensor(lens, dtype=I32, device=dev)
    rows = torch.randn(total, 576, generator=g).bfloat16().to(dev)
    rda.rda_mla_append_q4(rows, cache, table, kl, cu)
    out = rda.rda_mla_read_q4(cache, table, kl, total, cu)
    assert torch.equal(out[:, 512:], rows[:, 512:])
    # half a step of a group is at most 2^e, where the largest is at least 3.5 2^e
    x, y = rows[:, :512].float().reshape(-1, 16, 32), out[:, :512].float().reshape(-1, 16, 32)
    assert bool(((x - y).abs().amax(-1) <= x.abs().amax(-1) / 3.5).all())
    for n in (0, seqs // 2, seqs - 1):      # and some of them byte for byte
        for i in list(range(cu[n], cu[n + 1]))[-3:]:
            pos = i - cu[n]
            got = cache[int(table[n, pos // page]), pos % page].cpu()
            assert torch.equal(got, ref.encode_row(rows[i, :512].double().cpu(), rows[i, 512:].cpu()))
