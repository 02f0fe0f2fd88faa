"""Block-scaled caches on the GPU (gdn_cache_write, gdn_cache_read) against the MX
encoders of inputs.py, bit for bit: codes, scales, and the values read back."""
import numpy as np
import pytest
import torch

from gated_deltanet_scan_amd import api, inputs

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def make(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def encoded(x, fp4):
    """(codes, scales, values) of x on the host, as bytes."""
    c, s, v = (inputs.to_mxfp4 if fp4 else inputs.to_mxfp8)(x.float().cpu().numpy())
    return torch.from_numpy(c), torch.from_numpy(s), torch.from_numpy(v)


def filled(lead, H, D, fp4, seed=0):
    """A cache that holds something everywhere, so that a stray write shows."""
    c = api.cache_empty(*lead, H=H, D=D, fp4=fp4)
    g = torch.Generator().manual_seed(seed)
    for t in c:
        t.view(torch.uint8).copy_(torch.randint(100, 120, t.shape, generator=g, dtype=torch.uint8))
    return c


def raw(c):
    return [t.view(torch.uint8).cpu() for t in c]


FORMATS = pytest.mark.parametrize("fp4", [True, False], ids=["fp4", "fp8"])
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


@FORMATS
@TYPES
@pytest.mark.parametrize("H,D", [(1, 32), (3, 64), (2, 128), (16, 128)])
def test_packed_ragged(H, D, dtype, fp4):
    """Sequences of one token to several workgroups, of none, and of more than their slot takes."""
    new, size, use = [1, 300, 0, 5, 40, 7], [10, 1000, 4, 5, 33, 50], [3, 777, 2, 5, 20, 0]
    gap = 6                                                 # places of no sequence between the slots
    cu_new = np.concatenate([[0], np.cumsum(new)])
    cu_k = np.concatenate([[0], np.cumsum(size)])
    k, v = (make((cu_new[-1], H, D), dtype, s, 2.0) for s in (1, 2))
    cache = filled((int(cu_k[-1]) + gap,), H, D, fp4)
    want, before = raw(cache), raw(cache)
    for i, x in ((0, k), (2, v)):
        c, s, _ = encoded(x, fp4)
        for q in range(len(new)):
            for t in range(new[q]):
                p = use[q] - new[q] + t
                if 0 <= p < size[q]:
                    want[i][cu_k[q] + p], want[i + 1][cu_k[q] + p] = c[cu_new[q] + t], s[cu_new[q] + t]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    kw = dict(k_len=dev(use), cu_k=dev(cu_k), max_k=max(size))
    api.cache_write(k.cuda(), v.cuda(), *cache, cu_new=dev(cu_new), max_new=max(new), **kw)
    for a, b in zip(raw(cache), want):
        assert torch.equal(a, b)
    # and read back: the places in use, nothing else
    shape = (int(cu_k[-1]) + gap, H, D)
    out = [torch.full(shape, 99.0, dtype=dtype, device="cuda") for _ in range(2)]
    got = api.cache_read(*cache, k=out[0], v=out[1], **kw)
    for i in range(2):
        assert got[i] is out[i]
        ref = torch.full(shape, 99.0, dtype=F32)
        vals = values(want[2 * i], want[2 * i + 1], fp4)
        for q in range(len(new)):
            n = min(use[q], size[q])
            ref[cu_k[q]:cu_k[q] + n] = vals[cu_k[q]:cu_k[q] + n]
        assert torch.equal(out[i].cpu().float(), ref)


@FORMATS
def test_thousands_of_sequences(fp4):
    """Many packed sequences, no bound on their lengths given: a bound of all tokens."""
    n, H, D = 20000, 1, 32
    r = np.random.default_rng(5)
    new, size = r.integers(0, 3, n), r.integers(0, 6, n)
    cu_new, cu_k = (np.concatenate([[0], np.cumsum(x)]) for x in (new, size))
    k = make((cu_new[-1], H, D), BF, 1)
    cache = filled((int(cu_k[-1]),), H, D, fp4)
    want = raw(cache)
    c, s, _ = encoded(k, fp4)
    c = c.view(torch.uint8)
    token = np.arange(cu_new[-1])
    seq = np.searchsorted(cu_new, token, side="right") - 1
    place = size[seq] - new[seq] + (token - cu_new[seq])
    at = torch.from_numpy((cu_k[seq] + place)[place >= 0])
    token = torch.from_numpy(token[place >= 0])
    for i in (0, 2):
        want[i][at], want[i + 1][at] = c[token], s[token]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    api.cache_write(k.cuda(), k.cuda(), *cache, cu_new=dev(cu_new), cu_k=dev(cu_k))
    for a, b in zip(raw(cache), want):
        assert torch.equal(a, b)
    got = api.cache_read(*cache, cu_k=dev(cu_k), dtype=F32)
    for t, i in zip(got, (0, 2)):
        assert torch.equal(t.cpu(), values(want[i], want[i + 1], fp4))


def values(codes, scales, fp4):
    """What bytes stand for, from the formats' fields, on the host."""
    if fp4:
        mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])
        x = mag[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    else:
        x = codes.contiguous().view(F8).float()
    return (x.double() * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)).float()


@FORMATS
@TYPES
def test_every_magnitude(dtype, fp4):
    """Blocks of every exponent that the type has, rounding borders and both signs: codes, scales and values."""
    r = np.random.default_rng(3)
    e = torch.arange(-133 if dtype == BF else -149, 128).repeat_interleave(2)
    x = torch.from_numpy(r.uniform(-1, 1, (len(e), 1, 32)))
    mids = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.9]) / 8
    x[:, 0, :10] = mids * torch.where(torch.arange(len(e)) % 2 == 0, 1.0, -1.0)[:, None]
    x = (x * torch.exp2(e.double())[:, None, None]).to(dtype)
    x[torch.isinf(x)] = 0
    x[4] = 0
    x[5] = -0.0
    c, s, vals = encoded(x, fp4)
    cache = api.cache_empty(1, len(e), H=1, D=32, fp4=fp4)
    api.cache_write(x[None].cuda(), (-x)[None].cuda(), *cache)
    got = raw(cache)
    assert torch.equal(got[1][0], s) and torch.equal(got[0][0], c.view(torch.uint8))
    k, v = api.cache_read(*cache, dtype=F32)
    assert torch.equal(k[0].cpu(), vals) and torch.equal(v[0].cpu(), -vals)
    kb, _ = api.cache_read(*cache)
    big = vals.abs().amax(-1) >= 2.0 ** -110                   # bf16 has every value there
    assert torch.equal(kb[0].cpu()[big].float(), vals[big])
    assert torch.all((kb[0].cpu().double() - vals.double()).abs() <= 2.0 ** -133)


@FORMATS
@TYPES
def test_not_finite(dtype, fp4):
    """A block with an infinity or a NaN reads as NaN, its neighbours as they are."""
    x = make((1, 3, 2, 128), dtype, 5)
    ref = encoded(x, fp4)[2]
    x[0, 0, 0, 33], x[0, 1, 1, 127], x[0, 2, 0, 0] = float("nan"), float("inf"), float("-inf")
    cache = api.cache_empty(1, 3, H=2, D=128, fp4=fp4)
    api.cache_write(x.cuda(), x.cuda(), *cache)
    for t in api.cache_read(*cache, dtype=F32):
        t = t.cpu()
        bad = torch.zeros_like(t, dtype=torch.bool)
        bad[0, 0, 0, 32:64] = bad[0, 1, 1, 96:] = bad[0, 2, 0, :32] = True
        assert torch.isnan(t[bad]).all() and torch.equal(t[~bad], ref[~bad])
    assert int((cache[1] == 255).sum()) == 3


@FORMATS
def test_batched_views(fp4):
    """[B, n, H, D] and [B, F, N, H, D] tokens, slices of a fused projection, slots with room, single places."""
    B, room, H, D = 3, 50, 2, 64
    fused = make((B, 6, 3, H, D), BF, 8).cuda()
    k, v = fused[:, :, 1], fused[:, :, 2]
    whole = filled((B, room), H, D, fp4)
    part = [t[:, :20] for t in whole]
    want = raw(whole)
    for i, x in ((0, k), (2, v)):
        c, s, _ = encoded(x, fp4)
        want[i][:, 14:20], want[i + 1][:, 14:20] = c.view(torch.uint8), s
    api.cache_write(k, v, *part)                                # no k_len: the last places of the 20
    for a, b in zip(raw(whole), want):
        assert torch.equal(a, b)
    got = api.cache_read(*part, dtype=F32)
    assert got[0].shape == (B, 20, H, D) and got[0].is_contiguous()
    for t, i in zip(got, (0, 2)):
        assert torch.equal(t.cpu(), values(want[i], want[i + 1], fp4)[:, :20])
    # frames, and per-slot lengths
    frames = filled((B, room), H, D, fp4)
    n = torch.tensor([6, 50, 11], dtype=torch.int32, device="cuda")
    api.cache_write(k.reshape(B, 2, 3, H, D), v.reshape(B, 2, 3, H, D), *frames, k_len=n)
    kr, _ = api.cache_read(*frames, dtype=F32, k_len=n)
    for b, m in enumerate(n.tolist()):
        assert torch.equal(kr[b, m - 6:m].cpu(), encoded(k[b], fp4)[2])
    # one place a slot
    one = [t[:, :1] for t in whole]
    api.cache_write(k[:, -1:], v[:, -1:], *one)
    kr, vr = api.cache_read(*one, dtype=F32)
    assert torch.equal(kr.cpu(), encoded(k[:, -1:], fp4)[2]) and torch.equal(vr.cpu(), encoded(v[:, -1:], fp4)[2])


@FORMATS
def test_lengths_outside_the_slot(fp4):
    """Negative, zero and too long lengths on the device: tokens outside the slot are dropped, reads stop at it."""
    B, L, H, D = 4, 8, 1, 32
    n = torch.tensor([-3, 0, 10, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    cache = filled((B, L), H, D, fp4)
    want = raw(cache)
    k = make((B, 4, H, D), BF, 1)
    c, s, _ = encoded(k, fp4)
    want[0][2, 6:], want[1][2, 6:] = c.view(torch.uint8)[2, :2], s[2, :2]      # places 6 .. 9 of 8
    want[2][2, 6:], want[3][2, 6:] = want[0][2, 6:], want[1][2, 6:]
    api.cache_write(k.cuda(), k.cuda(), *cache, k_len=n)
    for a, b in zip(raw(cache), want):
        assert torch.equal(a, b)
    out = torch.full((B, L, H, D), 5.0, device="cuda")
    api.cache_read(*cache, k_len=n, k=out, v=torch.empty_like(out))
    assert torch.all(out[:2] == 5) and torch.equal(out[2:].cpu(), values(want[0], want[1], fp4)[2:])


def test_refusals():
    c = api.cache_empty(2, 8, H=2, D=64, fp4=True)
    k = make((2, 3, 2, 64), BF, 0).cuda()
    with pytest.raises(ValueError, match="alike"):
        api.cache_write(k, k[:, :2], *c)
    with pytest.raises(ValueError, match="batch"):
        api.cache_write(k[:1], k[:1], *c)
    with pytest.raises(TypeError, match="float8"):
        api.cache_read(c[0].float(), *c[1:])
    with pytest.raises(ValueError, match="shape"):
        api.cache_read(c[0], c[1][:, :4], c[2], c[3])
    with pytest.raises(ValueError, match="equally"):
        api.cache_read(c[0][:, :4], c[1][:, :4].contiguous(), c[2][:, :4], c[3][:, :4])
    with pytest.raises(ValueError, match="packed"):
        api.cache_write(k[0], k[0], *c, cu_new=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="evenly"):
        api.cache_write(k.transpose(1, 2), k.transpose(1, 2), *api.cache_empty(2, 8, H=3, D=64, fp4=True))


@FORMATS
def test_layers_side_by_side_are_refused(fp4):
    """One layer of a packed [T, layers, H, X] cache, with bounds that its tokens' distance passes: nothing is
    written or read."""
    T, layers, H, D = 12, 8, 2, 64
    whole = filled((T, layers), H, D, fp4)
    before = raw(whole)
    one = [t[:, 3] for t in whole]
    cu = torch.tensor([0, 4, 12], dtype=torch.int32, device="cuda")
    new = make((T, H, D), BF, 1).cuda()
    fwd = api.attention_fwd_fp4 if fp4 else api.attention_fwd_fp8
    with pytest.raises(ValueError, match="packed tokens"):
        api.cache_write(new, new, *one, cu_new=cu, max_new=8, max_k=8)
    with pytest.raises(ValueError, match="packed tokens"):
        api.cache_read(*one, cu_k=cu, max_k=8)
    with pytest.raises(ValueError, match="packed tokens"):
        fwd(new, *one, cu_q=cu, max_q=8, max_k=8)
    for a, b in zip(raw(whole), before):
        assert torch.equal(a, b)
