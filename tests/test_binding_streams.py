"""Which stream's memory a call of the binding uses (CPU: the allocator, the
streams and the library are stand-ins).  A call with stream=s takes what it
makes for itself from s's pool: a block of the current stream's pool may still
be in use by that stream's earlier calls, which s does not wait for, and a
temporary given back to that pool could be overwritten before s has read it."""
import contextlib
import types

import pytest
import torch

from gated_delta_amd import rda

DEV = torch.device("cuda", 0)


class Gpu(torch.Tensor):
    """A host tensor that says it is on the GPU."""
    device = property(lambda self: DEV)

    def record_stream(self, stream):
        self.__dict__.setdefault("on", []).append(stream)


def gpu(t):
    return t.as_subclass(Gpu)


class FakeStream:
    def __init__(self, name, device=DEV):
        self.name, self.device, self.cuda_stream = name, device, id(self)


class FakeTorch:
    """torch, with allocations on the GPU noted with the stream current then."""

    def __init__(self):
        self.current, self.made = FakeStream("current"), []
        self.cuda = types.SimpleNamespace(
            stream=self.stream, current_stream=lambda dev=None: self.current,
            current_device=lambda: 0, set_device=lambda i: None)

    def __getattr__(self, name):
        return getattr(torch, name)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        try:
            yield
        finally:
            self.current = before

    def note(self, t):
        self.made.append((t, self.current))
        return t

    def empty(self, *shape, dtype, device):
        assert device == DEV
        return self.note(gpu(torch.zeros(*shape, dtype=dtype)))

    def from_numpy(self, x):
        return types.SimpleNamespace(to=lambda dev: self.note(gpu(torch.from_numpy(x))))


class FakeLib:
    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096
        return lambda *a: 5 if name == "rda_max_chunks" else 0


@pytest.fixture
def fake(monkeypatch):
    t = FakeTorch()
    monkeypatch.setattr(rda, "torch", t)
    monkeypatch.setattr(rda, "_load", FakeLib)
    monkeypatch.setattr(rda, "_raw_stream", None)
    yield t
    for f in (rda.rda_mla_decode_workspace_bytes, rda.rda_verify_drafts_workspace_bytes):
        f.cache_clear()


def bf(*shape):
    return gpu(torch.zeros(*shape, dtype=torch.bfloat16))


def f32(*shape):
    return gpu(torch.zeros(*shape))


def ints(*values):
    return gpu(torch.tensor(values, dtype=torch.int32))


TABLE = gpu(torch.zeros(2, 3, dtype=torch.int32))

CALLS = {
    "mla_prefill": lambda s: rda.rda_mla_prefill(bf(6, 2, 192), bf(8, 2, 256), bf(8, 64), 0.1, [0, 2, 6],
                                                 [0, 3, 8], want_lse=True, stream=s),
    "mla_decode": lambda s: rda.rda_mla_decode(bf(2, 1, 4, 576), bf(6, 8, 576), TABLE, ints(5, 7), 0.1,
                                               want_lse=True, stream=s),
    "mla_append": lambda s: rda.rda_mla_append(bf(3, 576), bf(6, 8, 576), TABLE, ints(5, 7), [0, 1, 3], stream=s),
    "verify_drafts": lambda s: rda.rda_verify_drafts(f32(2, 3, 9), f32(2, 2, 9),
                                                     gpu(torch.zeros(2, 2, dtype=torch.int32)), f32(2, 3), stream=s),
}
MADE = {"mla_prefill": 4, "mla_decode": 3, "mla_append": 1, "verify_drafts": 3}


def mixer(*lead):
    """q, k, v, a, b of the mixer."""
    return [bf(*lead, 128) for _ in range(3)] + [f32(*lead), f32(*lead)]


def diag(*lead):
    return [bf(*lead, 128) for _ in range(3)] + [f32(*lead, 128), f32(*lead)]


RAW = [bf(4, 2, 128) for _ in range(3)] + [f32(3, 2, 128, 4), f32(4, 2), f32(4, 2)]
CU = [0, 1, 6]
CALLS.update({
    "prefill": lambda s: rda.rda_prefill(*mixer(6, 2), CU, stream=s),
    "prefill_norm_gate": lambda s: rda.rda_prefill_norm_gate(*mixer(6, 2), bf(6, 2, 128), CU, stream=s),
    "prefill_diag": lambda s: rda.rda_prefill_diag(*diag(6, 2), cu_seqlens=CU, stream=s),
    "decode_step": lambda s: rda.rda_decode_step(*mixer(3, 2), f32(3, 2, 128, 128), stream=s),
    "decode_step_diag": lambda s: rda.rda_decode_step_diag(*diag(3, 2), f32(3, 2, 128, 128), stream=s),
    "decode_tokens": lambda s: rda.rda_decode_tokens(*mixer(3, 4, 2), f32(3, 2, 128, 128), stream=s),
    "decode_tokens_diag": lambda s: rda.rda_decode_tokens_diag(*diag(3, 4, 2), f32(3, 2, 128, 128), stream=s),
    "output_norm_gate": lambda s: rda.rda_output_norm_gate(f32(5, 128), bf(5, 128), stream=s),
    "prologue": lambda s: rda.rda_prologue(*RAW, cu_seqlens=[0, 3, 4], stream=s),
    "decode_step_prologue": lambda s: rda.rda_decode_step_prologue(*RAW, f32(4, 2, 128, 128), stream=s),
    "chunk_table": lambda s: rda.rda_chunk_table(ints(*CU), 2, 6, device=DEV, stream=s),
})
MADE.update(prefill=4, prefill_norm_gate=4, prefill_diag=4, decode_step=1, decode_step_diag=1, decode_tokens=1,
            decode_tokens_diag=1, output_norm_gate=1, prologue=6, decode_step_prologue=1, chunk_table=3)


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_the_launch_stream(fake, name):
    s = FakeStream("side")
    out = CALLS[name](s)
    assert len(fake.made) == MADE[name]
    assert all(stream is s for _, stream in fake.made), [x.name for _, x in fake.made]
    # what the caller gets is kept from reuse until the caller's stream is past it too
    made = [t for t, _ in fake.made]
    for t in out if isinstance(out, tuple) else (out,):
        if any(t is m for m in made):
            assert t.__dict__.get("on") == [fake.current]


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_the_current_stream(fake, name):
    CALLS[name](None)
    assert len(fake.made) == MADE[name]
    assert all(stream is fake.current for _, stream in fake.made)


@pytest.mark.parametrize("name", ["mla_prefill", "mla_decode", "mla_append", "verify_drafts"])
def test_stream_of_another_device_is_refused(fake, name):
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](FakeStream("other", torch.device("cuda", 1)))
