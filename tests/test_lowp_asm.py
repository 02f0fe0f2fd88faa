"""The gfx950 assembly of the low-precision kernels, on the host.

Spills in a loop that holds matrix instructions, and loops over a buffer
descriptor's values, cost the kernels most of their speed.  The product's tiles
load memory straight to LDS with waits of their own: the compiler must add none
for these loads (it would wait for all of them before every read of LDS), and the
loads of a block stand before the barrier at which they are counted.
"""
import os
import re
import shutil
import subprocess

import pytest

from gated_deltanet_scan_amd import build
from test_ops_asm_loops import blocks_of, looped_spills, reach


def compiled(name, tmp):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not shutil.which(hipcc) and not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    out = tmp / "k.s"
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    r = subprocess.run([hipcc, *flags, "-I", os.path.join(build.ROOT, "include"), "--cuda-device-only", "-S",
                        os.path.join(build.PKG, "csrc", name), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return out.read_text()


def kernels(text, pattern):
    return {m.group(1): m.group(0)
            for m in re.finditer(r"^(_Z\w*(?:%s)\w*):.*?^\.Lfunc_end" % pattern, text, re.S | re.M)}


@pytest.fixture(scope="module")
def attention(tmp_path_factory):
    found = kernels(compiled("gdn_attn_mx.hip", tmp_path_factory.mktemp("mx")), "attn_fwd_kernel|attn_few_kernel")
    assert len(found) == 2 * (4 + 6), list(found)             # formats; tiles, and head sizes by row tiles
    return found


@pytest.fixture(scope="module")
def products(tmp_path_factory):
    found = kernels(compiled("gdn_matmul.hip", tmp_path_factory.mktemp("mm")), "matmul_kernel|matmul_few_kernel")
    assert len(found) == 4 + 2, list(found)
    return found


def test_no_spills_in_the_loops(attention, products):
    for name, body in {**attention, **products}.items():
        texts, after = blocks_of(body)
        assert any("v_mfma" in t and b in reach(after, b) for b, t in enumerate(texts)), name   # the loop is found
        assert not looped_spills(texts, after), name


def test_no_descriptor_loops(attention, products):
    for name, body in {**attention, **products}.items():
        for block in re.split(r"^\.LBB\w+:", body, flags=re.M):
            assert not (block.count("v_readfirstlane_b32") >= 4 and "s_and_saveexec" in block and
                        "buffer_load" in block), name


def test_no_packed_fp32(attention, products):
    for name, body in {**attention, **products}.items():
        assert not re.search(r"v_pk_(add|mul|fma)_f32", body), name


def test_tiles_wait_where_they_say(products):
    """In the block that holds a tile's products: every load to LDS stands before the one
    barrier, and nothing else waits for memory."""
    seen = 0
    for name, body in products.items():
        if "few" in name:
            continue
        wide = [t for t in blocks_of(body)[0] if t.count("v_mfma") >= 8]
        assert len(wide) == 1, name
        text = wide[0]
        assert text.count("s_barrier") == 1
        before, after = text.split("s_barrier")
        assert len(re.findall(r"buffer_load_dword\w* .*lds", before)) >= 4 and "buffer_load" not in after, name
        waits = re.findall(r"s_waitcnt[^\n]*vmcnt\((\d+)\)", text)
        assert len(waits) == 1, (name, waits)                   # the kernel's own
        assert text.count("v_mfma") == len(re.findall(r"v_mfma_f32_16x16x128_f8f6f4", text))
        seen += 1
    assert seen == 4


def test_tiles_end_with_no_load_under_way(products):
    """Loads to LDS run ahead past the last tile; a workgroup's LDS is another's once it ends."""
    tiles = {n: b for n, b in products.items() if "few" not in n}
    assert len(tiles) == 4
    for name, body in tiles.items():
        end = body[:body.rindex("s_endpgm")]
        lines = [t for t in (x.strip() for x in end.splitlines()) if t and not t.startswith((";", ".LBB"))]
        assert lines[-1] == "s_waitcnt vmcnt(0)", (name, lines[-3:])
