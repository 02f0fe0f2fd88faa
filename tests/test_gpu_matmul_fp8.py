"""Products of 8-bit floats on the GPU (gdn_matmul_fp8) against the fp64 oracle.

Tolerances.  The matrix instruction adds its 128 products eight at a time, each of
the eight cut at 2^-13 of the largest (so by less than 2^-13 of it), the sums of
eight in at least 24 bits: within a block the sum is off by at most
    7 2^-13 sum over eights of max |p|  +  16 u sum |p|,   u = 2^-24.
The scales' product and its use are three fp32 operations a block, the blocks are
added in fp32 (kb additions at most), and the output rounds once to bf16:
    e <= sum over blocks xs ws (that) + (kb + 4) u sum |x w| + 2^-8 |y| .
As a whole the error is one of rounding: relative to the norm of y at most
2^-8 / sqrt(3) = 2.26e-3 (half a step, evenly spread, at the lower end of a binade).
"""
import numpy as np
import pytest
import torch

from gated_deltanet_scan_amd import api, inputs
from oracle import ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def host(t):
    return t.detach().double().cpu().numpy()


def make(M, N, K, seed=0, spread=0):
    """Activations and weights as a block has them; spread: their exponents differ by up to so many bits."""
    g = torch.Generator().manual_seed(seed)
    x, w = torch.randn((M, K), generator=g), torch.randn((N, K), generator=g) * K ** -0.5
    if spread:
        x = x * torch.exp2(torch.randint(0, spread, (M, K), generator=g).float())
    xq = api.quantize_fp8(x.cuda())
    wq = inputs.to_fp8_weight(w.cuda())
    return (*xq, *wq)


def bars(x, xs, w, ws):
    M, K = x.shape
    N = w.shape[0]
    kb = xs.shape[1]
    val, cut, size = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    wr = ops.expand(ws, N, 0)
    for b in range(kb):
        sc = xs[:, b:b + 1] * wr[:, b][None, :]
        xb, wb = x[:, 128 * b:128 * (b + 1)], w[:, 128 * b:128 * (b + 1)]
        val += sc * (xb @ wb.T)
        size += sc * (np.abs(xb) @ np.abs(wb).T)
        for e in range(0, xb.shape[1], 8):
            p = np.abs(xb[:, None, e:e + 8] * wb[None, :, e:e + 8])
            cut += sc * p.max(-1)
    return val, 7 * 2.0 ** -13 * cut + (20 + kb) * U * size + 2.0 ** -8 * np.abs(val)


SHAPES = [(1, 1, 16), (1, 16, 128), (7, 96, 144), (16, 128, 128), (17, 130, 160), (33, 257, 400), (64, 64, 1040),
          (65, 48, 2048), (100, 200, 272), (129, 127, 112), (250, 300, 256), (5, 1000, 1040)]


@pytest.mark.parametrize("spread", [0, 10])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%dx%d" % s)
def test_product(shape, spread):
    x, xs, w, ws = make(*shape, seed=sum(shape), spread=spread)
    y = api.matmul_fp8(x, xs, w, ws)
    assert y.shape == shape[:2] and y.dtype == BF
    ref, bar = bars(host(x), host(xs), host(w), host(ws))
    err = np.abs(host(y) - ref)
    print("max err %.2e, most of the bar %.3f" % (err.max(), (err / (bar + 1e-300)).max()))
    assert np.all(err <= bar)
    if shape[0] * shape[1] >= 4096 and not spread:
        assert np.linalg.norm(host(y) - ref) <= 2.0 ** -8 / 3 ** 0.5 * np.linalg.norm(ref)


@pytest.mark.parametrize("M,N,K", [(880, 2048, 2048), (1777, 1000, 1040), (3000, 2304, 4096), (513, 6144, 2048),
                                   (5, 6144, 2048), (31, 8192, 2048), (64, 2048, 8192), (300, 512, 8192),
                                   # every kernel with several tiles to a workgroup, rows of one block and of less
                                   (66000, 512, 128), (70001, 264, 48), (9000, 2048, 144), (33, 40000, 16),
                                   (520, 16384, 128), (1000, 9000, 272),
                                   # many tokens and few columns: rows of workgroups of the kernels for few tokens
                                   (1777, 48, 1040), (4001, 16, 400), (100, 1000, 272), (201, 500, 2048)])
def test_large_products(M, N, K):
    """Against 64 bits on the card; the bound of the whole, and every element within 40 roundings of the typical
    value's: 8 bits of sum|p| 2^-13 7 / 8 are far below."""
    x, xs, w, ws = make(M, N, K, seed=M)
    y = api.matmul_fp8(x, xs, w, ws).double()
    xv = x.double() * xs.double().repeat_interleave(128, 1)[:, :K]
    wv = w.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    ref = xv @ wv.t()
    err = (y - ref).abs()
    assert err.norm() <= 2.0 ** -8 / 3 ** 0.5 * ref.norm()
    size = xv.abs() @ wv.abs().t()
    # max over eight <= their sum
    assert torch.all(err <= 7 * 2.0 ** -13 * size + (24 + K // 128) * U * size + 2.0 ** -8 * ref.abs())


def test_rows_and_blocks_are_told_apart():
    """Ones times ones: every output is the sum of its blocks' scales, which differ by row, column block and K block."""
    M, N, K = 70, 300, 400
    kb, nb = 4, 3
    x, w = torch.ones(M, K).to(F8).cuda(), torch.ones(N, K).to(F8).cuda()
    xs = torch.exp2(torch.arange(M * kb).reshape(M, kb) % 7 - 3.0).cuda()
    ws = torch.exp2(torch.arange(nb * kb).reshape(nb, kb) % 5 - 2.0).cuda()
    y = api.matmul_fp8(x, xs, w, ws)
    n = torch.tensor([128.0, 128.0, 128.0, 16.0], dtype=torch.float64)
    ref = ((xs.cpu().double() * n) @ ws.cpu().double().t()).repeat_interleave(128, 1)[:, :N]
    assert torch.equal(y.cpu(), ref.float().to(BF))


@pytest.mark.parametrize("M,H,D,C", [(5, 3, 32, 128), (70, 4, 64, 272), (300, 2, 16, 256), (17, 1, 5, 48)])
def test_parts(M, H, D, C):
    """q, k and v as three tensors hold what one product holds."""
    x, xs, w, ws = make(M, 3 * H * D, C, seed=M)
    one = api.matmul_fp8(x, xs, w, ws)
    three = api.matmul_fp8(x, xs, w, ws, parts=3)
    assert three.shape == (3, M, H * D)
    assert torch.equal(torch.cat(list(three), -1), one)


def test_views_streams_and_given_output():
    """Leading axes, a weight's rows from a larger tensor, a side stream, outputs that stay within their tensor."""
    x, xs, w, ws = make(30, 256, 256, seed=4)
    ref = api.matmul_fp8(x, xs, w, ws)
    y = api.matmul_fp8(x.view(2, 15, 256), xs.view(2, 15, 2), w, ws)
    assert torch.equal(y.view(30, 256), ref)
    half = api.matmul_fp8(x, xs, w[128:], ws[1:])
    assert torch.equal(half, ref[:, 128:])
    big = torch.full((32, 256), 7.0, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    api.matmul_fp8(x, xs, w, ws, y=big[1:31], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(big[1:31], ref) and torch.all(big[0] == 7) and torch.all(big[31] == 7)
    assert api.matmul_fp8(x[:0], xs[:0], w, ws).shape == (0, 256)


def test_not_finite():
    """A NaN code reaches its row (or column) alone; so does an infinite scale its block's."""
    x, xs, w, ws = make(40, 300, 256, seed=6)
    ref = api.matmul_fp8(x, xs, w, ws)
    x2 = x.clone()
    x2.view(torch.uint8)[3, 200] = 0x7F
    y = api.matmul_fp8(x2, xs, w, ws)
    keep = [i for i in range(40) if i != 3]
    assert torch.isnan(y[3]).all() and torch.equal(y[keep], ref[keep])
    w2 = w.clone()
    w2.view(torch.uint8)[255, 0] = 0xFF
    y = api.matmul_fp8(x, xs, w2, ws)
    keep = [i for i in range(300) if i != 255]
    assert torch.isnan(y[:, 255]).all() and torch.equal(y[:, keep], ref[:, keep])
    xs2 = xs.clone()
    xs2[5, 1] = float("inf")
    y = api.matmul_fp8(x, xs2, w, ws)
    keep = [i for i in range(40) if i != 5]
    assert not torch.isfinite(y[5]).any() and torch.equal(y[keep], ref[keep])
