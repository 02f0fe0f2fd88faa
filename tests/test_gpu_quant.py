"""8-bit activations on the GPU (gdn_quantize_fp8, gdn_rms_norm_fwd_fp8) against
the fp64 oracle (oracle/ops.py) and, where every step is one fp32 operation, bit for
bit against the same operations in torch on the host.

Tolerances of the norm.  u = 2^-24; S the additions on the longest path of a row's
sum (64 in a lane and 10 across lanes up to 16384 columns, C/256 + 10 beyond).  t
is off by u |t|, the sum of squares by (S + 3) u of itself, so its root's inverse by
(S + 3)/2 + 3 half steps, y by e = ((S + 3)/2 + 6) u |y|, the scale by
((S + 3)/2 + 8) u.  An e4m3 code is then off by half a step, 2^-4 of the value or
2^-10 below the least normal one (in units of the scale), so
    |code scale - y| <= max(2^-4 |y|, 2^-10 scale) + (S + 16) u |y| .
"""
import numpy as np
import pytest
import torch

from gated_deltanet_scan_amd import api
from oracle import ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def host(t):
    return t.detach().double().cpu().numpy()


def make(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def recipe(x):
    """gdn_quantize_fp8 in torch's fp32 on the host: the same operations."""
    rows, C = x.shape
    n = -(-C // 128)
    g = torch.zeros((rows, n * 128))
    g[:, :C] = x.float()
    g = g.reshape(rows, n, 128)
    top = g.abs().amax(-1).clamp_min(2.0 ** -100)
    codes = (g * torch.full_like(top, 448.0).div(top)[..., None]).to(F8).reshape(rows, n * 128)[:, :C]
    return codes.contiguous().view(torch.uint8), top / 448.0


SHAPES = [(1, 1), (3, 2), (5, 7), (4, 8), (2, 127), (2, 129), (7, 130), (1, 512), (2, 513), (9, 1001), (37, 1024),
          (8, 2048), (17, 2055), (130, 4096), (6, 4104), (5, 8191), (3, 16384), (3, 16385), (2, 40000), (1500, 96)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_quantise_is_the_recipe(shape, dtype):
    x = make(shape, dtype, sum(shape), std=3.0)
    x[0, 0] = 0.0
    y, s = api.quantize_fp8(x.cuda())
    want, scale = recipe(x)
    assert torch.equal(y.view(torch.uint8).cpu(), want) and torch.equal(s.cpu(), scale)


def test_quantise_ranges():
    """Zeros, tiny and huge groups, infinities and NaN, each in its own group."""
    x = torch.zeros(3, 7 * 128)
    x[:, 128:256] = make((3, 128), F32, 1, 1e-38)
    x[:, 256:384] = make((3, 128), F32, 2, 1e38)
    x[:, 384:512] = make((3, 128), F32, 3)
    x[:, 512:640] = make((3, 128), F32, 4)
    x[1, 400], x[1, 520] = float("inf"), float("nan")
    x[:, 640:768] = 1e-45
    y, s = api.quantize_fp8(x.cuda())
    v = y.float().cpu() * s.cpu().repeat_interleave(128, 1)
    assert not v[:, :128].any() and torch.isfinite(v[[0, 2]]).all()
    fine = v[:, 256:384].double()
    assert torch.all((fine - x[:, 256:384]).abs() <= 2.0 ** -4 * x[:, 256:384].abs() + 2.0 ** -10 * s.cpu()[:, 2:3])
    assert not torch.isfinite(v[1, 384:512]).any()                       # an infinity: its group
    assert torch.isnan(v[1, 520]) and torch.isfinite(v[1, 521:640]).all()  # a NaN: itself
    want, scale = recipe(x[[0, 2]])
    assert torch.equal(y.view(torch.uint8).cpu()[[0, 2]], want) and torch.equal(s.cpu()[[0, 2]], scale)


def check_norm(x, w, r, eps, got):
    y8, s, total = got
    rows, C = x.shape
    S = 74 if C <= 16384 else C / 256 + 10
    y, t = ops.rms_norm(host(x), None if w is None else host(w), None if r is None else host(r), eps)
    if r is not None:
        want = (x.float() + r.float()).to(x.dtype)
        assert torch.equal(total, want)                                  # one rounding of the sum
    scale = ops.group_scales(y)
    gs = host(s)
    assert np.all(np.abs(gs - scale) <= ((S + 3) / 2 + 8) * U * scale)
    v = host(y8) * ops.expand(gs, C, 1)
    bar = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * ops.expand(gs, C, 1)) + (S + 16) * U * np.abs(y)
    err = np.abs(v - y)
    print("most of the bar %.4f" % (err / (bar + 1e-300)).max(initial=0))
    assert np.all(err <= bar)


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32)], ids=["bf16", "bf16_wf32", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_norm(shape, types):
    rows, C = shape
    dtype, wt = types
    x, r = make(shape, dtype, rows + C).cuda(), make(shape, dtype, rows + C + 1).cuda()
    w = (1 + make((C,), F32, 7, 0.2)).to(wt).cuda()
    check_norm(x, w, r, 1e-6, api.rms_norm_fwd_fp8(x, w, r))
    check_norm(x, None, None, 1e-3, api.rms_norm_fwd_fp8(x, eps=1e-3))


@pytest.mark.parametrize("shape", [(5000, 1500), (4200, 2048), (600, 9001), (700, 16384)], ids=lambda s: "%dx%d" % s)
def test_norm_many_rows(shape):
    """More rows than the card takes at once, where other kernels than for few rows run; the sum in place of x."""
    x, r, w = make(shape, BF, 1).cuda(), make(shape, BF, 2).cuda(), (1 + make(shape[1:], BF, 3, 0.2)).cuda()
    ref = api.rms_norm_fwd_fp8(x, w, r)
    check_norm(x, w, r, 1e-6, ref)
    few = api.rms_norm_fwd_fp8(x[:9], w, r[:9])
    assert torch.equal(few[2], ref[2][:9])
    check_norm(x[:9], w, r[:9], 1e-6, few)
    got = api.rms_norm_fwd_fp8(x, w, r, total=x)
    assert got[2] is x and torch.equal(x, ref[2]) and torch.equal(got[1], ref[1])
    assert torch.equal(got[0].view(torch.uint8), ref[0].view(torch.uint8))


def test_norm_in_place_and_on_a_stream():
    """The sum in place of x or of the residual; a side stream; given outputs."""
    x, r, w = make((300, 2048), BF, 1).cuda(), make((300, 2048), BF, 2).cuda(), (1 + make((2048,), BF, 3, 0.1)).cuda()
    ref = api.rms_norm_fwd_fp8(x, w, r)
    a, b = x.clone(), r.clone()
    for got, total in ((api.rms_norm_fwd_fp8(a, w, r, total=a), a), (api.rms_norm_fwd_fp8(x, w, b, total=b), b)):
        assert got[2] is total and torch.equal(total, ref[2])
        assert torch.equal(got[0].view(torch.uint8), ref[0].view(torch.uint8)) and torch.equal(got[1], ref[1])
    y, s = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = api.rms_norm_fwd_fp8(x, w, r, y=y, y_scale=s, stream=side)
    q = api.quantize_fp8(ref[2], stream=side)
    torch.cuda.synchronize()
    assert got[0] is y and got[1] is s
    assert torch.equal(y.view(torch.uint8), ref[0].view(torch.uint8)) and torch.equal(s, ref[1])
    assert torch.equal(q[1].cpu(), recipe(ref[2].cpu())[1])


def test_norm_rows_of_no_use():
    """A row of zeros, one with a NaN, one with an infinity: the others as without them."""
    x = make((6, 700), BF, 5)
    ref = api.rms_norm_fwd_fp8(x.cuda())
    x[1], x[2, 3], x[4, 699] = 0, float("nan"), float("inf")
    y, s, _ = api.rms_norm_fwd_fp8(x.cuda())
    keep = [0, 3, 5]
    assert torch.equal(y.view(torch.uint8)[keep], ref[0].view(torch.uint8)[keep]) and torch.equal(s[keep], ref[1][keep])
    assert not y[1].float().any() and torch.isfinite(s[1]).all()
    assert torch.isnan(y[2].float()).all()
    assert torch.isnan(y[4, 699].float())


def test_empty_and_leading_axes():
    y, s, t = api.rms_norm_fwd_fp8(torch.zeros(0, 256, dtype=BF, device="cuda"))
    assert y.shape == (0, 256) and s.shape == (0, 2) and t is None
    x = make((2, 3, 200), BF, 9).cuda()
    y, s = api.quantize_fp8(x)
    assert y.shape == (2, 3, 200) and s.shape == (2, 3, 2)
    want, scale = recipe(x.cpu().reshape(6, 200))
    assert torch.equal(y.view(torch.uint8).cpu().reshape(6, 200), want) and torch.equal(s.cpu().reshape(6, 2), scale)
    with pytest.raises(ValueError, match="residual"):
        api.rms_norm_fwd_fp8(x, total=x)
    with pytest.raises(ValueError, match="contiguous"):
        api.quantize_fp8(x[..., :100])
