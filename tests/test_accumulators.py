"""The hand-placed registers of the latent-attention kernels (CPU: the sources
are compiled to assembly).  Sums live in accumulation registers, and M0 is set
for LDS transfers, by assembly statements whose values the compiler does not
know of.  A register of its own that it put there between two statements would
destroy them without a word, so the listing may name neither outside the
statements.  Nor may those kernels spill: what is left out of registers comes
back with waits that the transfers in flight do not reckon with."""
import concurrent.futures
import os
import re
import subprocess

import pytest

from gated_delta_amd import build

ACC = re.compile(r"\ba\d+\b|\ba\[|accvgpr")
M0 = re.compile(r"\bm0\b")


def stray(listing, pattern):
    """Instructions outside assembly statements that match, by function."""
    found, fn, inside = {}, None, False
    for line in listing.splitlines():
        if m := re.match(r"(\w+):", line):
            fn = m[1]
        if "#ASMSTART" in line:
            inside = True
        elif "#ASMEND" in line:
            inside = False
        elif not inside:
            code = line.split(";")[0].strip()
            if code and not code.startswith(".") and pattern.search(code):
                found.setdefault(fn, []).append(code)
    return found


def kernels(listing):
    """(name, spilled vector registers, bytes of scratch) of the kernels."""
    meta = listing[listing.index("amdhsa.kernels:"):]
    out = []
    for part in re.split(r"\n  - ", meta)[1:]:
        get = lambda key: re.search(rf"\.{key}:\s+(\S+)", part)[1]
        if ".vgpr_spill_count" in part:
            out.append((get("symbol"), int(get("vgpr_spill_count")), int(get("private_segment_fixed_size"))))
    return out


def users(word):
    out = []
    for path in build.sources():
        with open(path) as f:
            if re.search(word, f.read()):
                out.append(path)
    return out


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    where = tmp_path_factory.mktemp("asm")
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]

    def compile_one(path):
        out = str(where / (os.path.basename(path) + ".s"))
        subprocess.run([os.environ.get("HIPCC", "hipcc"), *flags, "--cuda-device-only", "-S", "-o", out, path],
                       check=True, capture_output=True)
        with open(out) as f:
            return f.read()

    paths = users(r"dma16_\w+|rda_mla_acc\.h")
    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        return dict(zip(paths, pool.map(compile_one, paths)))


def test_accumulation_registers(listings):
    paths = users(r"rda_mla_acc\.h")
    assert len(paths) == 2
    for path in paths:
        assert not stray(listings[path], ACC), path
        assert listings[path].count("v_mfma_f32_32x32x16_bf16 a[") > 0


def test_m0(listings):
    assert len(listings) == 3
    for path, text in listings.items():
        assert not stray(text, M0), path
        assert text.count("s_mov_b32 m0,") > 0


def test_no_spills(listings):
    for path in users(r"rda_mla_acc\.h"):
        found = kernels(listings[path])
        assert found
        for name, spilled, scratch in found:
            assert (spilled, scratch) == (0, 0), name


def test_what_the_listing_check_sees():
    text = """kernel_a:
	v_mov_b32_e32 v0, v1  ; a3 in a comment
	;;#ASMSTART
	v_accvgpr_write_b32 a[3], v0
	s_mov_b32 m0, s1
	;;#ASMEND
	s_barrier
kernel_b:
	v_accvgpr_read_b32 v1, a7
	buffer_load_dword a[4:7], v0, s[0:3], 0 offen
	s_mov_b32 m0, -1
	.amdhsa_accum_offset 256
"""
    assert stray(text, ACC) == {"kernel_b": ["v_accvgpr_read_b32 v1, a7",
                                             "buffer_load_dword a[4:7], v0, s[0:3], 0 offen"]}
    assert stray(text, M0) == {"kernel_b": ["s_mov_b32 m0, -1"]}
    meta = "amdhsa.kernels:\n  - .agpr_count: 0\n    .private_segment_fixed_size: 84\n    .symbol: k.kd\n    .vgpr_spill_count: 20\n"
    assert kernels(meta) == [("k.kd", 20, 84)]
