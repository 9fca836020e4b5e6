"""The hand-placed registers of rda_mla_decode_q4 (CPU: its listing), as in
test_accumulators: sums in a[0] .. a[63] and M0 are set by assembly statements
whose values the compiler does not know of.  The query's operands, which it does
know of, live in the accumulation registers above; nothing of its own may be
below, and no register that it spilled may come back inside the loop, where the
wait would be one for the transfers in flight."""
import os
import re
import subprocess

import pytest

from gated_delta_amd import build
from test_accumulators import M0, kernels, stray

BELOW_64 = re.compile(r"\ba([0-9]|[1-5][0-9]|6[0-3])\b|\ba\[([0-9]|[1-5][0-9]|6[0-3])[:\]]")


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    path = next(p for p in build.sources() if p.endswith("rda_mla_decode_q4.hip"))
    out = str(tmp_path_factory.mktemp("asm") / "q4.s")
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    subprocess.run([os.environ.get("HIPCC", "hipcc"), *flags, "--cuda-device-only", "-S", "-o", out, path],
                   check=True, capture_output=True)
    with open(out) as f:
        return f.read()


def loops(listing):
    """The bodies of the tile loops: between the first product into the sums and
    the settling wait behind the last, function by function."""
    out = {}
    for part in re.split(r"\n(?=_Z\w+:)", listing):
        m = re.match(r"(_Z\w+):", part)
        code = part.split("s_endpgm")[0]
        lines = code.splitlines()
        at = [i for i, x in enumerate(lines) if "v_mfma_f32_32x32x16_bf16 a[" in x]
        if m and at:
            out[m[1]] = lines
    return out


def test_registers(listing):
    assert not stray(listing, BELOW_64)
    assert not stray(listing, M0)
    assert listing.count("v_mfma_f32_32x32x16_bf16 a[") > 0 and listing.count("s_mov_b32 m0,") > 0


def test_no_scratch_beside_the_products(listing):
    """Neither a basic block with products nor one between two of them reads scratch."""
    found = loops(listing)
    assert len(found) == 2, list(found)
    for name, lines in found.items():
        at = [i for i, x in enumerate(lines) if "v_mfma_f32_32x32x16_bf16 a[" in x]
        # runs of products: the loop of a piece over a sequence, and over the prefix
        runs, start = [], at[0]
        for a, b in zip(at, at[1:]):
            if b - a > 1200:
                runs.append((start, a))
                start = b
        runs.append((start, at[-1]))
        assert len(runs) == 2, name
        for a, b in runs:
            code = [x.split(";")[0] for x in lines[a:b]]
            assert not [x for x in code if "scratch_" in x], name


def test_little_is_spilled(listing):
    for name, spilled, scratch in kernels(listing):
        assert spilled <= 16 and scratch <= 64, (name, spilled, scratch)
