"""The C ABI of the operators around the scan, on the host: bad calls are
rejected with the documented status before any launch.  The fake addresses are
never dereferenced.
"""
import ctypes
import os

import pytest
import torch

from gated_deltanet_scan_amd import _lib, api

OK, INVALID, UNSUPPORTED, ALIGN, ALIAS, WORKSPACE = 0, 1, 2, 3, 4, 5
BF16, F32 = _lib.GDN_BF16, _lib.GDN_F32
BASE = 0x7f0000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from gated_deltanet_scan_amd import build
        build.build()
    return _lib.load()


def addresses(names):
    return {n: BASE + i * (1 << 36) for i, n in enumerate(names)}


# ------------------------------------------------------------------ layer norm
def norm(rows=4, C=64, io=BF16, w=BF16, eps=1e-6):
    return _lib.GdnNormDesc(rows, C, io, w, eps)


NF = ["x", "w", "b", "y", "mean", "rstd"]
NB = ["dy", "x", "w", "mean", "rstd", "dx", "dw", "db", "ws"]


def norm_fwd(lib, d, **over):
    p = dict(addresses(NF), **over)
    return lib.gdn_layer_norm_fwd(None if d is None else ctypes.byref(d), *[p[n] for n in NF], None)


def norm_bwd(lib, d, ws_bytes=1 << 35, **over):
    p = dict(addresses(NB), **over)
    return lib.gdn_layer_norm_bwd(None if d is None else ctypes.byref(d), *[p[n] for n in NB], ws_bytes, None)


@pytest.mark.parametrize("d,expect", [
    (None, INVALID), (norm(rows=-1), INVALID), (norm(C=0), INVALID), (norm(eps=0.0), INVALID),
    (norm(eps=float("nan")), INVALID), (norm(eps=float("inf")), INVALID), (norm(io=_lib.GDN_FP8_E4M3), INVALID),
    (norm(io=F32, w=BF16), INVALID), (norm(C=(1 << 20) + 1), UNSUPPORTED),
])
def test_norm_descriptor(lib, d, expect):
    assert norm_fwd(lib, d) == expect and norm_bwd(lib, d) == expect


def test_norm_pointers(lib):
    d, a, b = norm(), addresses(NF), addresses(NB)
    assert norm_fwd(lib, d, x=None) == INVALID and norm_fwd(lib, d, y=None) == INVALID
    for n in ("dy", "x", "mean", "rstd", "dx"):
        assert norm_bwd(lib, d, **{n: None}) == INVALID, n
    assert norm_fwd(lib, d, x=a["x"] + 1) == ALIGN and norm_fwd(lib, d, mean=a["mean"] + 2) == ALIGN
    assert norm_fwd(lib, norm(w=F32), w=a["w"] + 2) == ALIGN
    assert norm_bwd(lib, d, dw=b["dw"] + 1) == ALIGN and norm_bwd(lib, d, ws=b["ws"] + 16) == ALIGN
    assert norm_fwd(lib, d, y=a["x"]) == ALIAS and norm_fwd(lib, d, rstd=a["mean"] + 12) == ALIAS
    assert norm_bwd(lib, d, dx=b["dy"]) == ALIAS and norm_bwd(lib, d, dw=b["ws"] + 256) == ALIAS
    need = lib.gdn_layer_norm_workspace_size(ctypes.byref(d))
    assert need == 2 * 64 * 4                                     # one row of partial sums for a few rows
    assert norm_bwd(lib, d, ws_bytes=need - 1) == WORKSPACE and norm_bwd(lib, d, ws=None) == WORKSPACE
    assert lib.gdn_layer_norm_workspace_size(ctypes.byref(norm(rows=0))) == 0
    assert norm_fwd(lib, norm(rows=0), x=None, y=None) == OK
    assert norm_bwd(lib, norm(rows=0), **{n: None for n in NB}) == OK


# ------------------------------------------------------------------ rotary
def rot(tokens=6, pos_rows=6, Hq=2, Hk=2, D=64, axes=(16, 24, 24), io=BF16, flags=0, theta=1e4, n=None):
    dims = (ctypes.c_int32 * 4)(*axes[:4])
    return _lib.GdnRotaryDesc(tokens, pos_rows, Hq, Hk, D, len(axes) if n is None else n, dims, io, flags, theta)


RN = ["q", "k", "pos", "qo", "ko"]


def rotary(lib, d, **over):
    p = dict(addresses(RN), **over)
    return lib.gdn_rotary(None if d is None else ctypes.byref(d), *[p[n] for n in RN], None)


@pytest.mark.parametrize("d,expect", [
    (None, INVALID), (rot(tokens=-1), INVALID), (rot(pos_rows=0), INVALID), (rot(Hq=-1), INVALID), (rot(D=0), INVALID),
    (rot(n=0), INVALID), (rot(n=5), INVALID), (rot(axes=(15, 17)), INVALID), (rot(axes=(32, 34)), INVALID),
    (rot(axes=(-2, 8)), INVALID), (rot(axes=(0,)), INVALID), (rot(io=9), INVALID), (rot(flags=8), INVALID),
    (rot(theta=0.0), INVALID), (rot(theta=float("nan")), INVALID), (rot(D=68), UNSUPPORTED), (rot(D=264), UNSUPPORTED),
    (rot(Hq=65537), UNSUPPORTED),
])
def test_rotary_descriptor(lib, d, expect):
    assert rotary(lib, d) == expect


def test_rotary_pointers(lib):
    a = addresses(RN)
    for n in RN:
        assert rotary(lib, rot(), **{n: None}) == INVALID, n
    for n in ("q", "k", "qo", "ko"):
        assert rotary(lib, rot(), **{n: a[n] + 8}) == ALIGN, n
    assert rotary(lib, rot(), pos=a["pos"] + 2) == ALIGN
    assert rotary(lib, rot(), qo=a["q"] + 16) == ALIAS            # in place exactly, or apart
    assert rotary(lib, rot(), qo=a["k"]) == ALIAS and rotary(lib, rot(), ko=a["qo"]) == ALIAS
    assert rotary(lib, rot(), ko=a["pos"]) == ALIAS
    assert rotary(lib, rot(tokens=0), **{n: None for n in RN}) == OK
    assert rotary(lib, rot(Hq=0, Hk=0), **{n: None for n in RN}) == OK


# ------------------------------------------------------------------ the torch side
def test_torch_refusals():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="device tensor"):
        api.layer_norm_fwd(x)
    with pytest.raises(ValueError, match="device tensor"):
        api.layer_norm_bwd(x, x, x[:, 0], x[:, 0])
    with pytest.raises(TypeError):
        api.layer_norm_fwd([1.0])
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="device tensor"):
        api.rotary(q, q, torch.zeros(4, 1, dtype=torch.int32), axes=(64,))
    with pytest.raises(TypeError):
        api.rotary(None, None, torch.zeros(4, 1, dtype=torch.int32), axes=(64,))


# ------------------------------------------------------------------ attention
def attn(tq=8, tk=8, qs=0, ks=0, vs=0, room=0, n=2, Hq=4, Hk=2, D=64, mq=4, mk=4, block=1, io=BF16, flags=0, scale=0.1):
    return _lib.GdnAttnDesc(tq, tk, qs, ks, vs, room, n, Hq, Hk, D, mq, mk, block, io, flags, scale)


AF = ["q", "k", "v", "cu_q", "cu_k", "k_len", "o", "lse", "ws"]
AB = ["q", "k", "v", "o", "lse", "dO", "cu_q", "cu_k", "dq", "dk", "dv", "ws"]


def attn_fwd(lib, d, ws_bytes=1 << 35, **over):
    p = dict(addresses(AF), cu_q=None, cu_k=None, k_len=None)
    p.update(over)
    return lib.gdn_attn_fwd(None if d is None else ctypes.byref(d), *[p[n] for n in AF], ws_bytes, None)


def attn_bwd(lib, d, ws_bytes=1 << 35, **over):
    p = dict(addresses(AB), cu_q=None, cu_k=None)
    p.update(over)
    return lib.gdn_attn_bwd(None if d is None else ctypes.byref(d), *[p[n] for n in AB], ws_bytes, None)


@pytest.mark.parametrize("d,expect", [
    (None, INVALID), (attn(n=-1), INVALID), (attn(Hq=0), INVALID), (attn(Hk=3), INVALID), (attn(D=0), INVALID),
    (attn(tq=-1), INVALID), (attn(mk=-1), INVALID), (attn(io=2), INVALID), (attn(flags=2), INVALID),
    (attn(flags=1, block=0), INVALID), (attn(scale=0.0), INVALID), (attn(scale=-1.0), INVALID),
    (attn(scale=float("nan")), INVALID), (attn(qs=248), INVALID), (attn(ks=120), INVALID), (attn(room=3), INVALID),
    (attn(tq=9), INVALID), (attn(mk=5), INVALID),              # uniform sequences must fill the tensors
    (attn(D=48), UNSUPPORTED), (attn(D=256), UNSUPPORTED), (attn(Hq=1 << 15, Hk=1 << 15), UNSUPPORTED),
    (attn(ks=(1 << 20) + 8), UNSUPPORTED), (attn(tq=1 << 32, mq=1 << 31 - 1, n=2), UNSUPPORTED),
])
def test_attn_descriptor(lib, d, expect):
    assert attn_fwd(lib, d) == expect and attn_bwd(lib, d) == expect


def test_attn_pointers(lib):
    d, a, b = attn(), addresses(AF), addresses(AB)
    for n in ("q", "k", "v", "o"):
        assert attn_fwd(lib, d, **{n: None}) == INVALID, n
        assert attn_fwd(lib, d, **{n: a[n] + 8}) == ALIGN, n
    for n in ("q", "k", "v", "o", "lse", "dO", "dq", "dk", "dv"):
        assert attn_bwd(lib, d, **{n: None}) == INVALID, n
    for n in ("q", "k", "v", "o", "dO", "dq", "dk", "dv"):
        assert attn_bwd(lib, d, **{n: b[n] + 8}) == ALIGN, n
    assert attn_fwd(lib, d, lse=a["lse"] + 2) == ALIGN and attn_fwd(lib, d, k_len=a["k_len"] + 1) == ALIGN
    assert attn_fwd(lib, attn(qs=260)) == ALIGN                     # 520 bytes: not a multiple of 16
    assert attn_bwd(lib, d, cu_q=b["cu_q"] + 2, cu_k=b["cu_k"]) == ALIGN
    assert attn_fwd(lib, d, o=a["q"]) == ALIAS and attn_fwd(lib, d, lse=a["o"] + 64) == ALIAS
    assert attn_fwd(lib, attn(ks=256), o=a["k"] + 7 * 512) == ALIAS  # inside the strided view's last row
    assert attn_fwd(lib, attn(room=100), o=a["v"] + 103 * 256) == ALIAS
    assert attn_fwd(lib, d, cu_q=a["o"]) == ALIAS
    assert attn_bwd(lib, d, dk=b["dv"]) == ALIAS and attn_bwd(lib, d, dq=b["dO"]) == ALIAS
    need = lib.gdn_attn_workspace_size_bwd(ctypes.byref(d))
    assert need == 256                                              # a float per query row
    assert attn_bwd(lib, d, ws_bytes=need - 1) == WORKSPACE and attn_bwd(lib, d, ws=None) == WORKSPACE
    assert attn_bwd(lib, d, dv=b["ws"]) == ALIAS and attn_bwd(lib, d, ws=b["ws"] + 16) == ALIGN


def test_attn_split_workspace(lib):
    # few queries against a long cache: fp32 partial outputs and one logarithm a row and split
    d = attn(tq=2, mq=1, tk=2 * 32768, mk=32768)
    need = lib.gdn_attn_workspace_size(ctypes.byref(d))
    rows = 2 * 4
    n = need // (rows * (64 + 1) * 4)
    assert n >= 8 and need == (n * rows * 64 * 4 + 255) // 256 * 256 + (n * rows * 4 + 255) // 256 * 256
    assert attn_fwd(lib, d, ws_bytes=need - 1) == WORKSPACE and attn_fwd(lib, d, ws=None) == WORKSPACE
    a = addresses(AF)
    assert attn_fwd(lib, d, ws=a["ws"] + 64) == ALIGN and attn_fwd(lib, d, lse=a["ws"] + 256) == ALIAS
    assert lib.gdn_attn_workspace_size(ctypes.byref(attn())) == 0
    assert lib.gdn_attn_workspace_size(None) == 0 and lib.gdn_attn_workspace_size_bwd(None) == 0


def test_attn_nothing_to_do(lib):
    none = {n: None for n in AF}
    assert attn_fwd(lib, attn(n=0, tq=0, tk=0), **none) == OK
    assert attn_fwd(lib, attn(tq=0, mq=0), **none) == OK
    assert attn_bwd(lib, attn(n=0, tq=0, tk=0), **{n: None for n in AB}) == OK


def test_attn_torch_refusals():
    q = torch.zeros(2, 5, 4, 64)
    with pytest.raises(ValueError, match="device tensor"):
        api.attention_fwd(q, q, q)
    with pytest.raises(ValueError, match="must be"):
        api.attention_fwd(q, q[0], q[0])
    with pytest.raises(ValueError, match="head size"):
        api.attention_fwd(q, q[..., :32], q[..., :32])
    with pytest.raises(TypeError):
        api.attention_fwd(q.half(), q.half(), q.half())


@pytest.mark.parametrize("scale,status", [(0.9e-30, INVALID), (1e-38, INVALID), (2e30, INVALID), (2e-30, None)])
def test_attn_range_of_scale(lib, scale, status):
    st = attn_fwd(lib, attn(scale=scale))
    assert st == status if status is not None else st != INVALID
