"""The binding of the 4-bit latent cache (CPU: the allocator, the streams and
the library are stand-ins): which stream's memory a call uses, and what may
serve as its workspace."""
import pytest
import torch

from gated_delta_amd import rda
from test_binding_streams import DEV, TABLE, FakeStream, bf, f32, fake, gpu, ints  # noqa: F401


def bytes_(*shape):
    return gpu(torch.zeros(*shape, dtype=torch.uint8))


CALLS = {
    "decode": lambda s, **kw: rda.rda_mla_decode_q4(bf(2, 1, 4, 576), bytes_(6, 8, 400), TABLE, ints(5, 7), 0.1,
                                                    want_lse=True, stream=s, **kw),
    "append": lambda s: rda.rda_mla_append_q4(bf(3, 576), bytes_(6, 8, 400), TABLE, ints(5, 7), [0, 1, 3], stream=s),
    "read": lambda s: rda.rda_mla_read_q4(bytes_(6, 8, 400), TABLE, ints(5, 7), 3, [0, 1, 3], stream=s),
}
MADE = {"decode": 3, "append": 1, "read": 2}


@pytest.fixture(autouse=True)
def forget_sizes():
    yield
    rda.rda_mla_decode_q4_workspace_bytes.cache_clear()


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_the_launch_stream(fake, name):  # noqa: F811
    rda.rda_mla_decode_q4_workspace_bytes.cache_clear()
    s = FakeStream("side")
    out = CALLS[name](s)
    assert len(fake.made) == MADE[name]
    assert all(stream is s for _, stream in fake.made), [x.name for _, x in fake.made]
    made = [t for t, _ in fake.made]
    for t in out if isinstance(out, tuple) else (out,):
        if any(t is m for m in made):
            assert t.__dict__.get("on") == [fake.current]


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_the_current_stream(fake, name):  # noqa: F811
    rda.rda_mla_decode_q4_workspace_bytes.cache_clear()
    CALLS[name](None)
    assert len(fake.made) == MADE[name]
    assert all(stream is fake.current for _, stream in fake.made)


@pytest.mark.parametrize("name", CALLS)
def test_stream_of_another_device_is_refused(fake, name):  # noqa: F811
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](FakeStream("other", torch.device("cuda", 1)))


def test_workspace(fake):  # noqa: F811
    rda.rda_mla_decode_q4_workspace_bytes.cache_clear()
    call = lambda w: CALLS["decode"](None, workspace=w)
    call(bytes_(4096))
    call(f32(1024))
    for bad in (torch.zeros(4096, dtype=torch.uint8), gpu(torch.zeros(1, dtype=torch.uint8).expand(4096)),
                bytes_(8192)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            call(bad)
    with pytest.raises(TypeError, match="workspace"):
        call(4096)


def test_shapes(fake):  # noqa: F811
    """Tables, lengths and offsets that do not belong together."""
    rda.rda_mla_decode_q4_workspace_bytes.cache_clear()
    cache, kv = bytes_(6, 8, 400), bf(3, 576)
    for call in (
        lambda: rda.rda_mla_append_q4(kv, cache, TABLE, ints(5), [0, 1, 3]),
        lambda: rda.rda_mla_append_q4(kv, cache, TABLE, ints(5, 7), [0, 3]),
        lambda: rda.rda_mla_append_q4(bf(3, 512), cache, TABLE, ints(5, 7), [0, 1, 3]),
        lambda: rda.rda_mla_append_q4(kv, bytes_(6, 8, 576), TABLE, ints(5, 7), [0, 1, 3]),
        lambda: rda.rda_mla_append_q4(kv, cache, TABLE, ints(5, 7), [0, 1, 3], weight=f32(576)),
        lambda: rda.rda_mla_read_q4(cache, TABLE, ints(5), 3, [0, 1, 3]),
        lambda: rda.rda_mla_read_q4(cache, TABLE, ints(5, 7), -1),
        lambda: rda.rda_mla_read_q4(cache, TABLE, ints(5, 7), 3, [0, 1, 3], out=bf(4, 576)),
        lambda: rda.rda_mla_read_q4(cache, ints(1, 2), ints(5, 7), 3, [0, 1, 3]),
        lambda: rda.rda_mla_decode_q4(bf(2, 1, 4, 512), cache, TABLE, ints(5, 7), 0.1),
        lambda: rda.rda_mla_decode_q4(bf(3, 1, 4, 576), cache, TABLE, ints(5, 7), 0.1),
        lambda: rda.rda_mla_decode_q4(bf(2, 1, 4, 576), cache, TABLE, ints(5, 7), 0.1, prefix_len=9),
        lambda: rda.rda_mla_decode_q4(bf(2, 1, 4, 576), cache, TABLE, ints(5, 7), 0.1, prefix_len=9,
                                      prefix_table=ints(3)),
    ):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        rda.rda_mla_append_q4(f32(3, 576), cache, TABLE, ints(5, 7), [0, 1, 3])
    with pytest.raises(TypeError):
        rda.rda_mla_decode_q4(bf(2, 1, 4, 576), bf(6, 8, 400), TABLE, ints(5, 7), 0.1)
