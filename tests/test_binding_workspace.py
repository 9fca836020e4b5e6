"""A workspace that a caller passes has to be memory that the kernels may
write from its first to its last byte (CPU: the library is a stand-in)."""
import pytest
import torch

import test_binding_streams as bs
from gated_delta_amd import rda
from test_binding_streams import bf, f32, fake, ints  # noqa: F401

CALLS = {
    "mla_decode": lambda w: rda.rda_mla_decode(bf(2, 1, 4, 576), bf(6, 8, 576), bs.TABLE, ints(5, 7), 0.1, workspace=w),
    "verify_drafts": lambda w: rda.rda_verify_drafts(
        f32(2, 3, 9), f32(2, 2, 9), bs.gpu(torch.zeros(2, 2, dtype=torch.int32)), f32(2, 3), workspace=w),
    "prefill": lambda w: rda.rda_prefill(*bs.mixer(6, 2), workspace=w),
    "prefill_norm_gate": lambda w: rda.rda_prefill_norm_gate(*bs.mixer(6, 2), bf(6, 2, 128), workspace=w),
    "prefill_diag": lambda w: rda.rda_prefill_diag(*bs.diag(6, 2), workspace=w),
}


@pytest.mark.parametrize("name", CALLS)
def test_workspace(fake, name):  # noqa: F811
    CALLS[name](bs.gpu(torch.zeros(4096, dtype=torch.uint8)))
    CALLS[name](f32(1024))
    with pytest.raises(ValueError, match="workspace"):
        CALLS[name](torch.zeros(4096, dtype=torch.uint8))             # host memory
    with pytest.raises(ValueError, match="workspace"):
        CALLS[name](bs.gpu(torch.zeros(1, dtype=torch.uint8).expand(4096)))   # one byte, seen 4096 times
    with pytest.raises(ValueError, match="workspace"):
        CALLS[name](bs.gpu(torch.zeros(8192, dtype=torch.uint8))[::2])
    with pytest.raises(TypeError, match="workspace"):
        CALLS[name](4096)
