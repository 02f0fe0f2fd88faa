"""The attention kernels' gfx950 assembly, on the host: no register is spilled in
any block of a loop that holds matrix instructions, its staging and masking
blocks included.  (At D = 128 the dk/dv kernel spills 23 registers around the
sums that it forms again element by element, after that loop.)
"""
import re

from test_ops_asm import kernels  # noqa: F401  (the fixture)


def blocks_of(body):
    """(texts, successors) of a kernel's basic blocks, in their order."""
    parts = re.split(r"^(\.LBB\w+):", body, flags=re.M)
    texts, place = [parts[0]] + parts[2::2], {name: i + 1 for i, name in enumerate(parts[1::2])}
    after = []
    for i, text in enumerate(texts):
        to = {place[b] for b in re.findall(r"^\s*s_c?branch\w*\s+(\.LBB\w+)", text, re.M)}
        ends = re.findall(r"^\s*(s_\w+)", text, re.M)
        if i + 1 < len(texts) and not (ends and ends[-1] in ("s_branch", "s_endpgm")):
            to.add(i + 1)
        after.append(to)
    return texts, after


def reach(after, start):
    seen, todo = set(), [start]
    while todo:
        for b in after[todo.pop()] - seen:
            seen.add(b)
            todo.append(b)
    return seen


def looped_spills(texts, after):
    """Blocks with spills that lie on a cycle through a block with products."""
    ways = [reach(after, b) for b in range(len(texts))]
    return [b for b, text in enumerate(texts) if "scratch_" in text and
            any("v_mfma" in texts[m] and m in ways[b] and b in ways[m] for m in range(len(texts)))]


def test_no_spills_in_the_loops(kernels):  # noqa: F811
    for name, body in kernels[0].items():
        texts, after = blocks_of(body)
        products = [b for b, text in enumerate(texts) if "v_mfma" in text and b in reach(after, b)]
        assert products, name                                  # the loop is found
        assert not looped_spills(texts, after), name


def test_a_spill_in_a_staging_block_is_found():
    loop = "k:\n{0}.LBB0_1:\n\tv_mfma_f32\n\ts_cbranch_scc0 .LBB0_3\n.LBB0_2:\n{1}\ts_branch .LBB0_1\n.LBB0_3:\n{2}\ts_endpgm\n"
    spill = "\tscratch_store_dword off, v0, s0\n"
    for at, found in ((0, []), (1, [2]), (2, [])):
        assert looped_spills(*blocks_of(loop.format(*[spill if i == at else "" for i in range(3)]))) == found
