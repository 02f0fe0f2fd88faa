"""Which views and sizes attention takes, on the host: the token stride that the
torch wrapper passes across the ABI (0 there means packed), and the ABI's own
bounds.
"""
import ctypes
import os

import pytest
import torch

from gated_deltanet_scan_amd import _lib, api


@pytest.mark.parametrize("one,shape", [
    ((1, 1, 4, 64), (8, 1, 4, 64)), ((1, 1, 1, 4, 64), (8, 1, 1, 4, 64)),        # single tokens
    ((1, 5, 4, 64), (8, 5, 4, 64)), ((1, 3, 5, 4, 64), (8, 3, 5, 4, 64)),        # whole sequences
    ((1, 1, 4, 64), (1, 5, 4, 64)), ((2, 1, 4, 64), (2, 5, 4, 64)), ((1, 4, 64), (6, 4, 64)),   # along the tokens
    ((2, 5, 1, 64), (2, 5, 4, 64)), ((2, 1, 1, 64), (2, 1, 4, 64)),              # along the heads
])
def test_broadcast_inputs_are_refused(one, shape):
    t = torch.zeros(one).expand(shape)
    with pytest.raises(ValueError, match="evenly spaced tokens"):
        api._token_strides(t, "q")


def test_overlapping_single_tokens_are_refused():
    t = torch.zeros(4096).as_strided((8, 1, 4, 64), (128, 256, 64, 1))            # tokens share half their heads
    with pytest.raises(ValueError, match="evenly spaced tokens"):
        api._token_strides(t, "q")


@pytest.mark.parametrize("shape", [(8, 1, 4, 64), (8, 1, 1, 4, 64), (2, 5, 4, 64), (2, 3, 5, 4, 64), (6, 4, 64)])
def test_views_that_are_taken(shape):
    H, D = shape[-2:]
    assert api._token_strides(torch.zeros(shape), "q") == (H * D, 0)
    fused = torch.zeros(shape[:-2] + (3 * H, D))[..., H:2 * H, :]
    assert api._token_strides(fused, "q") == (3 * H * D, 0)
    if len(shape) == 4:
        cache = torch.zeros((shape[0], 9) + shape[2:])[:, :shape[1]]
        want = (9 * H * D, 0) if shape[1] == 1 else (H * D, 9)
        assert api._token_strides(cache, "k") == want


# ------------------------------------------------------------------ the ABI's bounds
OK, INVALID, UNSUPPORTED, ALIAS = 0, 1, 2, 4
BASE = 0x7f0000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from gated_deltanet_scan_amd import build
        build.build()
    return _lib.load()


def both(lib, tq, tk, n, mq, mk, qs=0, ks=0, vs=0, room=0, Hq=4, Hk=2, D=64):
    """Statuses of the two passes on addresses that are no memory.  The outputs
    alias q, which is found last of all: what the ABI takes ends in ALIAS, and
    nothing is launched."""
    d = ctypes.byref(_lib.GdnAttnDesc(tq, tk, qs, ks, vs, room, n, Hq, Hk, D, mq, mk, 1, _lib.GDN_BF16, 0, 0.1))
    p = [BASE + i * (1 << 44) for i in range(9)]
    f = lib.gdn_attn_fwd(d, p[0], p[1], p[2], None, None, None, p[0], None, p[3], 1 << 40, None)
    b = lib.gdn_attn_bwd(d, p[0], p[1], p[2], p[4], p[5], p[6], None, None, p[0], p[7], p[8], p[3], 1 << 40, None)
    return f, b


@pytest.mark.parametrize("stride,tokens,most,expect", [
    (1 << 20, 4, 1, ALIAS), (1 << 20, 4, 2, ALIAS),
    ((1 << 20) + 8, 4, 2, UNSUPPORTED),                       # two tokens of one sequence that far apart
    ((1 << 20) + 8, 4, 1, ALIAS), (1 << 34, 4, 1, ALIAS),     # single tokens of a long cache's slots
    ((1 << 38) + 8, 4, 1, UNSUPPORTED),                       # past any tensor
])
@pytest.mark.parametrize("which", ["qs", "ks", "vs"])
def test_range_of_strides(lib, which, stride, tokens, most, expect):
    n = tokens // most
    assert both(lib, tokens, tokens, n, most, most, **{which: stride}) == (expect, expect)


# ------------------------------------------------------------------ launches
def test_launches_that_are_too_large_are_refused_first(lib):
    """2^32 work items in any of a call's launches: refused before the first."""
    n = 1 << 20
    assert both(lib, 16 * n, 16 * n, n, 16, 16, Hq=16, Hk=16, D=32) == (UNSUPPORTED, UNSUPPORTED)   # every launch
    assert both(lib, 16 * n, 0, n, 16, 0, Hq=16, Hk=16, D=32) == (UNSUPPORTED, UNSUPPORTED)         # o, dq
    assert both(lib, 0, 16 * n, n, 0, 16, Hq=16, Hk=16, D=32) == (OK, UNSUPPORTED)                  # dk and dv alone
    assert both(lib, 16 * n, 16 * n, n, 16, 16, Hq=15, Hk=15, D=32) == (ALIAS, ALIAS)               # just below


@pytest.mark.parametrize("Hq,Hk,D", [(4, 4, 64), (8, 1, 128), (6, 2, 16)])
@pytest.mark.parametrize("tq,tk", [(1, 20000), (700, 900), (3000, 40)])
def test_bounds_above_the_tensors_are_the_tensors(lib, Hq, Hk, D, tq, tk):
    """max_q and max_k only bound the lengths: whatever lies above the number of
    tokens is the same call, down to its splits and their workspace."""
    def sizes(mq, mk):
        d = ctypes.byref(_lib.GdnAttnDesc(tq, tk, 0, 0, 0, 0, 1, Hq, Hk, D, mq, mk, 1, _lib.GDN_BF16, 0, 0.1))
        return lib.gdn_attn_workspace_size(d), lib.gdn_attn_workspace_size_bwd(d)
    assert sizes((1 << 30) // Hq, 1 << 30) == sizes(tq, tk)
