"""Every kernel of gdn_matmul_fp8 and each way that it stores its outputs: whole lines within
one of the outputs, outputs past the first, and element by element where a tile ends
unevenly or lies in two of them.  SHAPES holds sizes that the rule of choice sends to each;
tests/test_matmul_rule.py asks the rule itself whether it does.

Tolerances are those of tests/test_gpu_matmul_fp8.py, formed on the card in 64 bits:
    7 2^-13 sum over blocks xs ws sum over eights of max |p| + (20 + kb) u sum |x w| + 2^-8 |y|.
"""
import pytest
import torch

from gated_deltanet_scan_amd import api, inputs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
UNITS = 256                                    # compute units of the card that the shapes are chosen for

# M, columns of one output, outputs, K
SHAPES = [
    (9, 20, 3, 272), (9, 21, 3, 144), (70, 334, 3, 1040), (70, 40, 3, 400),                    # up to 16 tokens a workgroup
    (100, 332, 3, 272), (100, 333, 3, 400), (201, 501, 1, 144),                                # up to 32
    (1777, 1001, 1, 400), (1777, 335, 3, 272), (1777, 344, 3, 144), (1777, 384, 3, 1040),      # 128 x 64
    (1777, 667, 3, 272), (1777, 664, 3, 400), (1777, 640, 3, 16), (1777, 2002, 1, 144),        # 128 x 128
    (1777, 1001, 3, 272), (1777, 1000, 3, 400), (1777, 1280, 3, 128), (1777, 2999, 1, 48),     # 256 x 128
    (7001, 683, 3, 272), (7001, 680, 3, 400), (7001, 512, 3, 144), (7001, 1999, 1, 16),        # 256 x 256
]
# one of each kernel, with tiles that end unevenly
EACH = [(9, 21, 3, 400), (100, 333, 3, 400), (1777, 335, 3, 400), (1777, 667, 3, 400), (1777, 1001, 3, 400),
        (7001, 683, 3, 400)]
ids = lambda s: "%dx%dx%dx%d" % s


def make(M, N, K, seed, spread=0):
    g = torch.Generator().manual_seed(seed)
    x, w = torch.randn((M, K), generator=g), torch.randn((N, K), generator=g) * K ** -0.5
    if spread:
        x = x * torch.exp2(torch.randint(0, spread, (M, K), generator=g).float())
    return (*api.quantize_fp8(x.cuda()), *inputs.to_fp8_weight(w.cuda()))


def one_tensor(y):
    """[parts, M, part] as [M, parts part]."""
    return y if y.dim() == 2 else y.transpose(0, 1).flatten(1)


def test_card():
    assert torch.cuda.get_device_properties(0).multi_processor_count == UNITS


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_every_element(shape):
    """Each element within its bar, operands of widely spread exponents; nothing written around the outputs; one
    tensor and several hold the same."""
    M, part, parts, K = shape
    N, kb = part * parts, -(-K // 128)
    x, xs, w, ws = make(M, N, K, M + N, spread=10)
    n = M * N
    room = torch.full((n + 4096,), 7.0, dtype=BF, device="cuda")
    y = room[2048:2048 + n].view((parts, M, part) if parts > 1 else (M, N))
    assert api.matmul_fp8(x, xs, w, ws, parts=parts, y=y) is y
    assert torch.all(room[:2048] == 7) and torch.all(room[2048 + n:] == 7)
    assert torch.equal(one_tensor(y), api.matmul_fp8(x, xs, w, ws))
    xd, wd = x.double(), w.double()
    wr = ws.double().repeat_interleave(128, 0)[:N]
    val, bar, size = (torch.zeros((M, N), dtype=torch.float64, device="cuda") for _ in range(3))
    for b in range(kb):
        sc = xs[:, b:b + 1].double() * wr[:, b][None, :]
        xb, wb = xd[:, 128 * b:128 * (b + 1)], wd[:, 128 * b:128 * (b + 1)].contiguous()
        val += sc * (xb @ wb.t())
        size += sc * (xb.abs() @ wb.abs().t())
        for e in range(0, xb.shape[1], 8):
            top = torch.zeros_like(val)
            for j in range(e, e + 8):
                top = torch.maximum(top, torch.outer(xb[:, j].abs(), wb[:, j].abs()))
            bar += 7 * 2.0 ** -13 * sc * top
    bar += (20 + kb) * U * size + 2.0 ** -8 * val.abs()
    err = (one_tensor(y).double() - val).abs()
    print("most of the bar %.3f" % float((err / (bar + 1e-300)).max()))
    assert torch.all(err <= bar)


@pytest.mark.parametrize("shape", EACH, ids=ids)
def test_rows_and_blocks_are_told_apart(shape):
    """Ones times ones: every output is the sum of its blocks' scales, which differ by row, column block and K block
    (powers of two, sums below 2^24 of their units, so exact before the one rounding to bf16)."""
    M, part, parts, K = shape
    N, kb = part * parts, -(-K // 128)
    nb = -(-N // 128)
    x, w = torch.ones(M, K).to(F8).cuda(), torch.ones(N, K).to(F8).cuda()
    xs = torch.exp2(torch.arange(M * kb).reshape(M, kb) % 7 - 3.0).cuda()
    ws = torch.exp2(torch.arange(nb * kb).reshape(nb, kb) % 5 - 2.0).cuda()
    n = torch.tensor([min(128, K - 128 * b) for b in range(kb)], dtype=torch.float64, device="cuda")
    ref = ((xs.double() * n) @ ws.double().t().contiguous()).repeat_interleave(128, 1)[:, :N].float().to(BF)
    assert torch.equal(one_tensor(api.matmul_fp8(x, xs, w, ws, parts=parts)), ref)


@pytest.mark.parametrize("shape", EACH, ids=ids)
def test_not_finite(shape):
    """A NaN code reaches its row (or column) alone, an infinite scale its row's block: rows and columns at the edges
    of tiles and inside them."""
    M, part, parts, K = shape
    N = part * parts
    x, xs, w, ws = make(M, N, K, 6)
    ref = one_tensor(api.matmul_fp8(x, xs, w, ws, parts=parts))
    rows = sorted({0, 3, min(63, M - 2), min(64, M - 2), M - 1})
    other = torch.ones(M, dtype=torch.bool, device="cuda")
    other[rows] = False
    x2 = x.clone()
    x2.view(torch.uint8)[rows, K - 1] = 0x7F
    y = one_tensor(api.matmul_fp8(x2, xs, w, ws, parts=parts))
    assert torch.isnan(y[~other]).all() and torch.equal(y[other], ref[other])
    xs2 = xs.clone()
    xs2[rows, 1] = float("inf")
    y = one_tensor(api.matmul_fp8(x, xs2, w, ws, parts=parts))
    assert not torch.isfinite(y[~other]).any() and torch.equal(y[other], ref[other])
    cols = sorted({0, 17, part - 1, min(part, N - 1), min(128, N - 1), N - 1})
    other = torch.ones(N, dtype=torch.bool, device="cuda")
    other[cols] = False
    w2 = w.clone()
    w2.view(torch.uint8)[cols, 0] = 0xFF
    y = one_tensor(api.matmul_fp8(x, xs, w2, ws, parts=parts))
    assert torch.isnan(y[:, ~other]).all() and torch.equal(y[:, other], ref[:, other])
