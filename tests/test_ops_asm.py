"""The attention kernels' gfx950 assembly, on the host.

Every matrix instruction takes one fragment from LDS (a 16-byte row read or a
pair of transposed reads) and the other from registers.  hipcc can sink LDS
reads whose first use lies past a later barrier below it, where other waves may
already overwrite the tile; counted between barriers, the reads of each basic
block must therefore cover its matrix instructions.  Spills and loops over a
buffer descriptor's values cost the kernels most of their speed, so neither may
appear there.
"""
import os
import re
import shutil
import subprocess

import pytest

from gated_deltanet_scan_amd import build

SRC = os.path.join(build.PKG, "csrc", "gdn_attn_bf16.hip")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not shutil.which(hipcc) and not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "attn.s"
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    r = subprocess.run([hipcc, *flags, "-I", os.path.join(build.ROOT, "include"), "--cuda-device-only", "-S", SRC,
                        "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = out.read_text()
    found = {m.group(1): m.group(0)
             for m in re.finditer(r"^(_ZN\w*attn_(?:fwd|dq|dkv)_kernel\w*):.*?^\.Lfunc_end", text, re.S | re.M)}
    assert len(found) == 4 + 3 + 3, list(found)
    return found, text


def test_reads_stay_with_their_products(kernels):
    bad = []
    for name, body in kernels[0].items():
        seen = 0
        for block in re.split(r"^\.LBB\w+:", body, flags=re.M):
            for part in block.split("s_barrier"):
                m = part.count("v_mfma_f32_32x32x16_bf16")
                seen += m
                if m and part.count("ds_read_b128") + part.count("ds_read_b64_tr_b16") / 2 < m:
                    bad.append((name, m))
        assert seen, name
    assert not bad


def test_no_spills_and_no_descriptor_loops(kernels):
    for name, body in kernels[0].items():
        for block in re.split(r"^\.LBB\w+:", body, flags=re.M):
            assert not ("v_mfma" in block and "scratch_" in block), name      # none where the products are
        # a loop over the values of a descriptor in vector registers reads them back lane by lane
        for block in re.split(r"^\.LBB\w+:", body, flags=re.M):
            assert not (block.count("v_readfirstlane_b32") >= 4 and "s_and_saveexec" in block and
                        "buffer_load" in block), name
