"""The C ABI and the torch side of the 8-bit projections, the block-scaled caches
and the attention over them, on the host: bad calls are rejected with the
documented status before any launch.  The fake addresses are never dereferenced.
"""
import ctypes
import os

import numpy as np
import pytest
import torch

from gated_deltanet_scan_amd import _lib, api, inputs

OK, INVALID, UNSUPPORTED, ALIGN, ALIAS, WORKSPACE = 0, 1, 2, 3, 4, 5
BF16, F32, FP8, FP4 = _lib.GDN_BF16, _lib.GDN_F32, _lib.GDN_FP8_E4M3, _lib.GDN_FP4_E2M1
BASE = 0x7f0000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from gated_deltanet_scan_amd import build
        build.build()
    return _lib.load()


def addresses(names):
    return {n: BASE + i * (1 << 36) for i, n in enumerate(names)}


def ref(d):
    return None if d is None else ctypes.byref(d)


# ------------------------------------------------------------------ norm and quantisation
def norm(rows=4, C=200, io=BF16, w=BF16, eps=1e-6):
    return _lib.GdnNormDesc(rows, C, io, w, eps)


RN, QN = ["x", "r", "w", "sum", "y", "ys"], ["x", "y", "ys"]


def rms(lib, d, **over):
    p = dict(addresses(RN), **over)
    return lib.gdn_rms_norm_fwd_fp8(ref(d), *[p[n] for n in RN], None)


def quant(lib, d, **over):
    p = dict(addresses(QN), **over)
    return lib.gdn_quantize_fp8(ref(d), *[p[n] for n in QN], None)


@pytest.mark.parametrize("d,expect", [
    (None, INVALID), (norm(rows=-1), INVALID), (norm(C=0), INVALID), (norm(io=FP8), INVALID),
    (norm(C=(1 << 20) + 1), UNSUPPORTED),
])
def test_quantise_descriptor(lib, d, expect):
    assert rms(lib, d) == expect and quant(lib, d) == expect


def test_norm_descriptor(lib):
    for d in (norm(eps=0.0), norm(eps=float("nan")), norm(eps=float("inf")), norm(io=F32, w=BF16), norm(w=9)):
        assert rms(lib, d) == INVALID


def test_quantise_pointers(lib):
    d, a, b = norm(), addresses(RN), addresses(QN)
    for n in ("x", "y", "ys"):
        assert rms(lib, d, **{n: None}) == INVALID and quant(lib, d, **{n: None}) == INVALID
    for n in ("x", "r", "w", "sum"):
        assert rms(lib, d, **{n: a[n] + 1}) == ALIGN, n
    assert rms(lib, d, ys=a["ys"] + 2) == ALIGN and quant(lib, norm(io=F32), x=b["x"] + 2) == ALIGN
    assert rms(lib, d, sum=a["x"] + 2) == ALIAS and rms(lib, d, sum=a["w"]) == ALIAS
    assert rms(lib, d, y=a["x"]) == ALIAS and rms(lib, d, y=a["r"] + 1599) == ALIAS
    assert rms(lib, d, ys=a["y"] + 796) == ALIAS and rms(lib, d, ys=a["sum"]) == ALIAS
    assert quant(lib, d, y=b["x"]) == ALIAS and quant(lib, d, ys=b["y"]) == ALIAS
    assert rms(lib, norm(rows=0), **{n: None for n in RN}) == OK
    assert quant(lib, norm(rows=0), **{n: None for n in QN}) == OK


# ------------------------------------------------------------------ products
def mm(M=5, N=96, K=160, parts=1):
    return _lib.GdnMatmulDesc(M, N, K, parts)


MN = ["x", "xs", "w", "ws", "y"]


def matmul(lib, d, **over):
    p = dict(addresses(MN), **over)
    return lib.gdn_matmul_fp8(ref(d), *[p[n] for n in MN], None)


@pytest.mark.parametrize("d,expect", [
    (None, INVALID), (mm(M=-1), INVALID), (mm(N=0), INVALID), (mm(K=0), INVALID), (mm(parts=0), INVALID),
    (mm(parts=5), INVALID), (mm(K=40), UNSUPPORTED), (mm(K=(1 << 20) + 16), UNSUPPORTED),
    (mm(N=(1 << 20) + 1), UNSUPPORTED), (mm(M=1 << 31), UNSUPPORTED), (mm(M=(1 << 31) - 1, N=1 << 20, K=16), UNSUPPORTED),
])
def test_matmul_descriptor(lib, d, expect):
    assert matmul(lib, d) == expect


def test_matmul_pointers(lib):
    d, a = mm(), addresses(MN)
    for n in MN:
        assert matmul(lib, d, **{n: None}) == INVALID, n
        assert matmul(lib, d, **{n: a[n] + 2}) == ALIGN, n
    assert matmul(lib, d, y=a["x"] + 784) == ALIAS and matmul(lib, d, y=a["ws"]) == ALIAS
    assert matmul(lib, d, y=a["w"] - 944) == ALIAS and matmul(lib, d, y=a["xs"]) == ALIAS
    assert matmul(lib, mm(M=0), **{n: None for n in MN}) == OK


# ------------------------------------------------------------------ caches
def cache(tn=8, tk=20, ks=0, vs=0, room=0, n=2, H=2, D=64, mn=4, mk=10, io=BF16, fmt=FP4):
    return _lib.GdnCacheDesc(tn, tk, ks, vs, room, n, H, D, mn, mk, io, fmt)


WN = ["k", "v", "cu_new", "cu_k", "k_len", "kc", "ks", "vc", "vs"]
RDN = ["kc", "ks", "vc", "vs", "cu_k", "k_len", "k", "v"]


def write(lib, d, **over):
    p = dict(addresses(WN), cu_new=None, cu_k=None, k_len=None)
    p.update(over)
    return lib.gdn_cache_write(ref(d), *[p[n] for n in WN], None)


def read(lib, d, **over):
    p = dict(addresses(RDN), cu_k=None, k_len=None)
    p.update(over)
    return lib.gdn_cache_read(ref(d), *[p[n] for n in RDN], None)


@pytest.mark.parametrize("d,expect", [
    (None, INVALID), (cache(n=-1), INVALID), (cache(H=0), INVALID), (cache(D=0), INVALID), (cache(tk=-1), INVALID),
    (cache(mk=-1), INVALID), (cache(io=FP8), INVALID), (cache(fmt=BF16), INVALID), (cache(room=9), INVALID),
    (cache(room=-1), INVALID), (cache(ks=120), INVALID), (cache(vs=-256), INVALID), (cache(mk=9), INVALID),
    (cache(D=16), UNSUPPORTED), (cache(D=48), UNSUPPORTED), (cache(H=1 << 15), UNSUPPORTED),
    (cache(tk=1 << 32, mk=1 << 31 - 1), UNSUPPORTED), (cache(room=1 << 31), UNSUPPORTED),
    (cache(ks=(1 << 31) + 8), UNSUPPORTED),
])
def test_cache_descriptor(lib, d, expect):
    assert write(lib, d) == expect and read(lib, d) == expect


def test_cache_pointers(lib):
    d, a, b = cache(), addresses(WN), addresses(RDN)
    assert write(lib, cache(tn=9)) == INVALID
    for n in ("k", "v", "kc", "ks", "vc", "vs"):
        assert write(lib, d, **{n: None}) == INVALID and read(lib, d, **{n: None}) == INVALID, n
    for n in ("k", "v", "kc", "vc"):
        assert write(lib, d, **{n: a[n] + 8}) == ALIGN and read(lib, d, **{n: b[n] + 8}) == ALIGN, n
    assert write(lib, d, k_len=a["k_len"] + 2) == ALIGN and read(lib, d, cu_k=b["cu_k"] + 1) == ALIGN
    assert write(lib, cache(ks=132)) == ALIGN                         # 264 bytes
    assert write(lib, d, ks=a["kc"] + 20 * 64 - 1) == ALIAS and write(lib, d, vc=a["kc"]) == ALIAS
    assert write(lib, d, kc=a["v"]) == ALIAS and write(lib, d, vs=a["ks"] + 79) == ALIAS
    assert write(lib, d, k_len=a["vs"]) == ALIAS
    assert write(lib, cache(room=50), vc=a["kc"] + 59 * 64) == ALIAS  # the second slot's last place
    assert write(lib, cache(ks=256), kc=a["k"] + 7 * 512 + 240) == ALIAS
    assert read(lib, d, k=b["vc"]) == ALIAS and read(lib, d, v=b["k"]) == ALIAS
    assert write(lib, cache(n=0, tn=0, tk=0), **{n: None for n in WN}) == OK
    assert write(lib, cache(tn=0, mn=0), **{n: None for n in WN}) == OK
    assert read(lib, cache(tk=0, mk=0), **{n: None for n in RDN}) == OK


# ------------------------------------------------------------------ attention
def test_workspace_of_loose_bounds(lib):
    """Many packed sequences whose lengths have no bound but the tensor's: chunks are a quarter of an even share of
    8192 at least, or as long as their offsets allow (2^31 bytes of codes, less four steps)."""
    for n, tk, Hq, Hk in ((1, 10 ** 9, 32, 8), (3000, 10 ** 7, 32, 8), (8, 2 ** 30, 128, 4), (100000, 10 ** 8, 8, 8)):
        d = _lib.GdnAttnDesc(n, tk, 0, 0, 0, 0, n, Hq, Hk, 128, 1, tk, 1, FP4, 1, 0.1)
        splits = 1 + max(4 * 8192 // (n * Hk), tk // (2 ** 31 // (Hk * 128) - 192))
        assert 0 <= lib.gdn_attn_workspace_size(ref(d)) <= splits * n * Hq * (128 + 1) * 4 + 512, (n, tk)


def attn(tq=8, tk=8, qs=0, ks=0, vs=0, room=0, n=2, Hq=4, Hk=2, D=64, mq=4, mk=4, block=1, io=FP4, flags=0, scale=0.1):
    return _lib.GdnAttnDesc(tq, tk, qs, ks, vs, room, n, Hq, Hk, D, mq, mk, block, io, flags, scale)


AN = ["q", "k", "ks", "v", "vs", "cu_q", "cu_k", "k_len", "o", "lse", "ws"]


def attn_mx(lib, d, fmt=FP4, ws_bytes=1 << 35, **over):
    p = dict(addresses(AN), cu_q=None, cu_k=None, k_len=None)
    p.update(over)
    fn = lib.gdn_attn_fwd_fp4 if fmt == FP4 else lib.gdn_attn_fwd_fp8
    return fn(ref(d), *[p[n] for n in AN], ws_bytes, None)


@pytest.mark.parametrize("fmt", [FP4, FP8])
def test_attention_descriptor(lib, fmt):
    def bad(**kw):
        return attn_mx(lib, attn(io=fmt, **kw), fmt)
    assert attn_mx(lib, None, fmt) == INVALID
    assert attn_mx(lib, attn(io=fmt), FP8 if fmt == FP4 else FP4) == INVALID     # each its own format
    for io in (BF16, F32):
        assert attn_mx(lib, attn(io=io), fmt) == INVALID
    assert bad(n=-1) == INVALID and bad(Hk=3) == INVALID and bad(scale=0.0) == INVALID and bad(tq=9) == INVALID
    assert bad(ks=120) == INVALID and bad(room=3) == INVALID and bad(flags=1, block=0) == INVALID
    assert bad(D=16) == UNSUPPORTED and bad(D=256) == UNSUPPORTED and bad(ks=256) == UNSUPPORTED
    assert bad(vs=256) == UNSUPPORTED
    # the calls that take bf16 and fp32 refuse it
    d = attn(io=fmt)
    a = [BASE + i * (1 << 36) for i in range(13)]
    assert lib.gdn_attn_fwd(ref(d), a[0], a[1], a[2], None, None, None, a[3], a[4], None, 0, None) == INVALID
    assert lib.gdn_attn_bwd(ref(d), *a[:6], None, None, *a[6:9], a[9], 1 << 35, None) == INVALID
    assert lib.gdn_attn_workspace_size_bwd(ref(d)) == 0


def test_attention_pointers(lib):
    d, a = attn(), addresses(AN)
    for n in ("q", "k", "ks", "v", "vs", "o"):
        assert attn_mx(lib, d, **{n: None}) == INVALID, n
    for n in ("q", "k", "v", "o"):
        assert attn_mx(lib, d, **{n: a[n] + 8}) == ALIGN, n
    assert attn_mx(lib, d, o=a["q"]) == ALIAS and attn_mx(lib, d, lse=a["o"] + 64) == ALIAS
    assert attn_mx(lib, d, o=a["k"] + 8 * 64 - 16) == ALIAS           # the codes' last bytes
    assert attn_mx(lib, d, lse=a["ks"] + 28) == ALIAS
    assert attn_mx(lib, attn(io=FP8), FP8, o=a["v"] + 8 * 128 - 16) == ALIAS
    assert attn_mx(lib, attn(room=100), o=a["v"] + 103 * 64) == ALIAS
    long = attn(tq=2, mq=1, tk=2 * 32768, mk=32768)
    need = lib.gdn_attn_workspace_size(ref(long))
    assert need > 0 and attn_mx(lib, long, ws_bytes=need - 1) == WORKSPACE and attn_mx(lib, long, ws=None) == WORKSPACE
    assert attn_mx(lib, long, ws=a["ws"] + 64) == ALIGN
    assert attn_mx(lib, attn(n=0, tq=0, tk=0), **{n: None for n in AN}) == OK


# ------------------------------------------------------------------ the torch side
def test_torch_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        api.rms_norm_fwd_fp8(x)
    with pytest.raises(ValueError, match="device tensor"):
        api.quantize_fp8(x)
    with pytest.raises(TypeError):
        api.quantize_fp8([1.0])
    w = torch.zeros(32, 64, dtype=torch.float8_e4m3fn)
    s = torch.zeros(4, 1)
    with pytest.raises(ValueError, match="parts"):
        api.matmul_fp8(w[:4], s, w, s[:1], parts=3)
    with pytest.raises(ValueError, match="device tensor"):
        api.matmul_fp8(w[:4], s, w, s[:1])
    with pytest.raises(ValueError, match="multiple of 32"):
        api.cache_empty(2, 8, H=2, D=48, fp4=True, device="cpu")
    for fp4, fwd in ((True, api.attention_fwd_fp4), (False, api.attention_fwd_fp8)):
        c = api.cache_empty(2, 8, H=2, D=64, fp4=fp4, device="cpu")
        assert c[0].shape == (2, 8, 2, 32 if fp4 else 64) and c[1].shape == (2, 8, 2, 2)
        with pytest.raises(ValueError, match="device tensor"):
            api.cache_write(torch.zeros(2, 1, 2, 64), torch.zeros(2, 1, 2, 64), *c)
        with pytest.raises(ValueError, match="device tensor"):
            api.cache_read(*c)
        with pytest.raises(ValueError, match="device tensor"):
            fwd(torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16), *c)
    with pytest.raises(TypeError, match="uint8"):
        api.cache_read(torch.zeros(2, 8, 2, 64), c[1], c[2], c[3])


def test_packed_tokens_of_a_cache():
    c = torch.zeros(3, 10, 2, 32, dtype=torch.uint8)
    assert api._packed_tokens(c, "k") == 0 and api._packed_tokens(c[:, :4], "k") == 10
    assert api._packed_tokens(c[:, :1], "k") == 10 and api._packed_tokens(c[:1, :1], "k") in (0, 10)
    both = torch.zeros(3, 10, 2, 2, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="packed"):
        api._packed_tokens(both[:, :, 0], "k")                       # k and v side by side in one tensor
    with pytest.raises(ValueError, match="evenly|packed"):
        api._packed_tokens(c[:, ::2], "k")
    s = torch.zeros(3, 10, 2, 1, dtype=torch.uint8)                  # one scale a row
    assert api._packed_tokens(s[:, :4], "k_scale") == 10


@pytest.mark.parametrize("name,tensor", [
    ("one of 32 layers", torch.zeros(16, 32, 2, 64, dtype=torch.uint8)[:, 3]),
    ("k beside v", torch.zeros(16, 2, 2, 32, dtype=torch.uint8)[:, 0]),
    ("every fourth token", torch.zeros(64, 2, 32, dtype=torch.uint8)[::4]),
    ("scales of one byte a row", torch.zeros(16, 4, 1, 1, dtype=torch.uint8)[:, 1]),
], ids=lambda x: x if isinstance(x, str) else "")
def test_tokens_of_a_packed_cache_lie_side_by_side(name, tensor):
    """[T, H, X] has no slots: tokens further apart than a row are no cache."""
    with pytest.raises(ValueError, match="packed tokens"):
        api._packed_tokens(tensor, "k")


def test_slots_of_one_place():
    """[B, 1, H, X] and [B, 1, 1, H, X] of longer slots, and packed tokens from the middle of a tensor, are caches."""
    c = torch.zeros(3, 10, 2, 32, dtype=torch.uint8)
    assert api._packed_tokens(c[:, 4:5], "k") == 10 and api._packed_tokens(c[:, 4:5, None], "k") == 10
    assert api._packed_tokens(c[1], "k") == 0 and api._packed_tokens(c[1, 3:7], "k") == 0


def test_weight_encoder():
    """The recipe: block maxima become +-448, values are within half a step."""
    r = np.random.default_rng(0)
    w = torch.from_numpy(r.standard_normal((200, 300)).astype(np.float32))
    w[128:, 256:] = 0
    codes, scale = inputs.to_fp8_weight(w)
    assert codes.shape == (200, 300) and scale.shape == (2, 3)
    v = codes.double() * scale.double().repeat_interleave(128, 0)[:200].repeat_interleave(128, 1)[:, :300]
    assert torch.all((v - w).abs() <= (w.abs() * 2.0 ** -4).clamp_min(float(scale.max()) * 2.0 ** -10) * (1 + 1e-6))
    assert codes[:128, :128].float().abs().max() == 448 and not codes[128:, 256:].float().any()
