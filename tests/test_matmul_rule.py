"""Which kernels of gdn_matmul_fp8 the GPU tests' sizes reach, on the host: the rule of
choice is plain C++, compiled here, so a later rule cannot leave a kernel untested."""
import os
import shutil
import subprocess

import pytest

from gated_deltanet_scan_amd import build
from test_gpu_matmul_tiles import EACH, SHAPES, UNITS

KINDS = 6
TILE = {2: 128, 3: 128, 4: 256, 5: 256}              # columns of a tile of kinds 2 to 5, which come through LDS

MAIN = """
#include "gdn_matmul_rule.hpp"
#include <cstdio>
int main() {
    long long m;
    int n, units;
    while (scanf("%lld %d %d", &m, &n, &units) == 3) printf("%d\\n", (int)gdnmatmul::choose(m, n, units));
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++") or shutil.which("amdclang++")
    if not cxx:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("rule")
    (at / "main.cpp").write_text(MAIN)
    exe = str(at / "main")
    subprocess.run([cxx, "-std=c++17", "-I", os.path.join(build.PKG, "csrc"), str(at / "main.cpp"), "-o", exe],
                   check=True)

    def ask(sizes):
        text = "".join("%d %d %d\n" % (m, n, UNITS) for m, n in sizes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [int(k) for k in out.split()]
    return ask


def stores(kind, part, parts):
    """Ways that a size's outputs are stored: in whole lines ("whole", and "later" where that is another output than
    the first), element by element ("single"), as the kernels decide for each tile."""
    N, found = part * parts, set()
    if kind < 2:
        return {"whole" if part % 4 == 0 else "single"} | ({"later"} if parts > 1 and part % 4 == 0 else set())
    for n0 in range(0, N, TILE[kind]):
        last = min(n0 + TILE[kind], N) - 1
        if n0 // part == last // part and part % 8 == 0:
            found |= {"whole"} | ({"later"} if n0 >= part else set())
        else:
            found.add("single")
    return found


def test_every_kernel_and_store_is_reached(choose):
    reached = {k: set() for k in range(KINDS)}
    for (M, part, parts, _), kind in zip(SHAPES, choose([(m, p * n) for m, p, n, _ in SHAPES])):
        reached[kind] |= stores(kind, part, parts)
    assert all(s == {"whole", "later", "single"} for s in reached.values()), reached


def test_every_kernel_is_reached_by_the_exact_tests(choose):
    kinds = choose([(m, p * n) for m, p, n, _ in EACH])
    assert kinds == list(range(KINDS))
    assert all("single" in stores(k, p, n) for k, (_, p, n, _) in zip(kinds, EACH))


def test_few_tokens_take_the_first_kernel(choose):
    sizes = [(m, n) for m in (1, 7, 16) for n in (1, 96, 6144, 1 << 20)]
    assert choose(sizes) == [0] * len(sizes)
