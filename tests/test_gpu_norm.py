"""Layer norm on the GPU (gdn_layer_norm_fwd, gdn_layer_norm_bwd) against the
fp64 oracle (oracle/ops.py).

Tolerances.  u = 2^-24 is fp32's half step, t the output type's (2^-8 for
bf16, 2^-24 for fp32), S the number of additions on the longest path of a
row's sum: at most 64 in a lane plus 10 across lanes up to 16384 columns,
C/256 + 10 beyond.  The mean is then off by at most S u <|x|>, h by
e_h = rstd S u <|x|> + (S + 4) u |h| (the variance's sum has S additions of
non-negative terms, so rstd is off by at most S/2 + 3 half steps), and
    y:  |w| e_h + 3 u (|h w| + |b|) + t |y|
    dx: rstd (4 u |g| + S u <|g|> + |h| (S u <|g h|> + <|g| e_h>) + e_h |<g h>|) + (S + 8) u |dx| + t |dx|
A column's sum has at most rows/(4 groups) + groups/16 + 12 additions, R:
    dw: sum |dy| e_h + R u sum |dy h| + t |dw|,   db: R u sum |dy| + t |db|.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_scan_amd import api, autograd
from oracle import ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def host(t):
    return t.detach().double().cpu().numpy()


def make(rows, C, dtype, wdtype, seed=0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, C), generator=g) + 0.5 * torch.randn((1, C), generator=g) + mean
    dy = torch.randn((rows, C), generator=g)
    w, b = 1 + 0.2 * torch.randn(C, generator=g), 0.2 * torch.randn(C, generator=g)
    return (x.to(dtype).cuda(), dy.to(dtype).cuda(), w.to(wdtype).cuda(), b.to(wdtype).cuda())


def check(got, ref, bar, name):
    if got.size == 0:
        assert got.shape == ref.shape
        return
    err = np.abs(got - ref)
    print("%s: max err %.3e, most of the bar %.3f" % (name, err.max(), (err / (bar + 1e-300)).max()))
    assert np.all(err <= bar), name


def bars(x, dy, w, b, eps, dtype, wdtype):
    rows, C = x.shape
    S = 74 if C <= 16384 else C / 256 + 10
    h, _, rstd = ops.layer_norm(x, eps=eps)
    rstd = rstd[:, None]
    mean = lambda a: a.mean(-1, keepdims=True)
    eh = rstd * S * U * mean(np.abs(x)) + (S + 4) * U * np.abs(h)
    y = ops.layer_norm(x, w, b, eps)[0]
    w1 = np.ones(C) if w is None else np.abs(w)
    b1 = np.zeros(C) if b is None else np.abs(b)
    by = w1 * eh + 3 * U * (np.abs(h) * w1 + b1) + T[dtype] * np.abs(y)
    dx, dw, db = ops.layer_norm_bwd(dy, x, w, eps)
    g = dy * (1 if w is None else w)
    ag = np.abs(g)
    bdx = (rstd * (4 * U * ag + S * U * mean(ag) + np.abs(h) * (S * U * mean(ag * np.abs(h)) + mean(ag * eh)) +
                   eh * np.abs(mean(g * h))) + (S + 8) * U * np.abs(dx) + T[dtype] * np.abs(dx))
    groups = max(1, min(1024, rows // 16 if C <= 4096 else rows // 4))
    R = rows / groups + groups / 16 + 16
    bdw = (np.abs(dy) * eh).sum(0) + R * U * np.abs(dy * h).sum(0) + T[wdtype] * np.abs(dw)
    bdb = R * U * np.abs(dy).sum(0) + T[wdtype] * np.abs(db)
    return (y, dx, dw, db), (by, bdx, bdw, bdb)


SHAPES = [(1, 1), (3, 2), (5, 7), (1, 64), (2, 513), (9, 1001), (37, 1024), (64, 2048), (17, 2055), (130, 4096),
          (6, 4104), (5, 8191), (3, 16384), (3, 16385), (2, 40000), (1500, 96)]
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)]


@pytest.mark.parametrize("types", TYPES, ids=["bf16", "bf16_wf32", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_forward_and_backward(shape, types):
    rows, C = shape
    dtype, wdtype = types
    eps = 1e-5
    x, dy, w, b = make(rows, C, dtype, wdtype, seed=rows + C)
    y, mean, rstd = api.layer_norm_fwd(x, w, b, eps=eps)
    dx, dw, db = api.layer_norm_bwd(dy, x, mean, rstd, w, b)
    torch.cuda.synchronize()
    assert dw.dtype == wdtype and db.dtype == wdtype and y.dtype == dtype and dx.dtype == dtype
    refs, bar = bars(host(x), host(dy), host(w), host(b), eps, dtype, wdtype)
    for got, r, t, n in zip((y, dx, dw, db), refs, bar, ("y", "dx", "dw", "db")):
        check(host(got), r, t, n)


@pytest.mark.parametrize("which", ["none", "weight", "bias"])
def test_optional_parameters(which):
    x, dy, w, b = make(50, 300, torch.bfloat16, torch.float32, seed=3)
    w, b = (w if which == "weight" else None), (b if which == "bias" else None)
    y, mean, rstd = api.layer_norm_fwd(x, w, b)
    dx, dw, db = api.layer_norm_bwd(dy, x, mean, rstd, w, b)
    torch.cuda.synchronize()
    assert (dw is None) == (w is None) and (db is None) == (b is None)
    refs, bar = bars(host(x), host(dy), None if w is None else host(w), None if b is None else host(b), 1e-6,
                     torch.bfloat16, torch.float32)
    for got, r, t, n in zip((y, dx, dw, db), refs, bar, ("y", "dx", "dw", "db")):
        if got is not None:
            check(host(got), r, t, n)


def test_large_mean_and_constant_rows():
    """A mean 300 times the spread (the two sums lose nothing to <x^2> - mu^2),
    and rows that do not vary: h = 0, y = bias exactly."""
    x, dy, w, b = make(20, 500, torch.float32, torch.float32, seed=4, mean=300.0)
    x[7] = 2.0
    y, mean, rstd = api.layer_norm_fwd(x, w, b)
    dx, dw, db = api.layer_norm_bwd(dy, x, mean, rstd, w, b)
    torch.cuda.synchronize()
    refs, bar = bars(host(x), host(dy), host(w), host(b), 1e-6, torch.float32, torch.float32)
    keep = np.arange(20) != 7
    check(host(y)[keep], refs[0][keep], bar[0][keep], "y")
    check(host(dx)[keep], refs[1][keep], bar[1][keep], "dx")
    check(host(dw), refs[2], bar[2], "dw")
    assert torch.equal(y[7], b)


def test_no_rows_and_a_bad_row():
    x, dy, w, b = make(4, 100, torch.bfloat16, torch.bfloat16)
    y, mean, rstd = api.layer_norm_fwd(x[:0], w, b)
    dx, dw, db = api.layer_norm_bwd(dy[:0], x[:0], mean, rstd, w, b)
    torch.cuda.synchronize()
    assert y.shape == (0, 100) and not dw.any() and not db.any()
    # a NaN or infinity stays in its own row
    x[1, 5], x[2, 99] = float("nan"), float("inf")
    y, _, _ = api.layer_norm_fwd(x, w, b)
    torch.cuda.synchronize()
    assert torch.isfinite(y[[0, 3]]).all() and not torch.isfinite(y[[1, 2]]).any()


def test_same_bits_every_time_and_in_a_graph():
    x, dy, w, b = make(3000, 2048, torch.bfloat16, torch.bfloat16, seed=6)
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    y, mean, rstd = api.layer_norm_fwd(x, w, b)
    outs = api.layer_norm_bwd(dy, x, mean, rstd, w, b)
    torch.cuda.synchronize()
    y2, m2, r2 = torch.empty_like(y), torch.empty_like(mean), torch.empty_like(rstd)
    o2 = [torch.empty_like(t) for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.layer_norm_fwd(x, w, b, y=y2, mean=m2, rstd=r2)
        api.layer_norm_bwd(dy, x, m2, r2, w, b, dx=o2[0], dweight=o2[1], dbias=o2[2], workspace=ws)
    for _ in range(3):
        for t in (y2, m2, r2, *o2):
            t.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        for a, c in zip((y, mean, rstd, *outs), (y2, m2, r2, *o2)):
            assert torch.equal(a, c)


def test_side_stream():
    x, dy, w, b = make(500, 1024, torch.bfloat16, torch.bfloat16, seed=8)
    ref = api.layer_norm_fwd(x, w, b)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = api.layer_norm_fwd(x, w, b, stream=s)[0]
    s.synchronize()
    assert torch.equal(y, ref)


def test_autograd():
    x, dy, w, b = make(4 * 30, 257, torch.bfloat16, torch.float32, seed=9)
    x, dy = x.reshape(4, 30, 257), dy.reshape(4, 30, 257)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    y = autograd.layer_norm(*leaves, eps=1e-5)
    y.backward(dy.transpose(0, 1).contiguous().transpose(0, 1))      # a gradient of another layout
    y0, mean, rstd = api.layer_norm_fwd(x, w, b, eps=1e-5)
    ref = api.layer_norm_bwd(dy, x, mean, rstd, w, b)
    torch.cuda.synchronize()
    assert torch.equal(y, y0)
    for a, r in zip(leaves, ref):
        assert torch.equal(a.grad, r)


def test_gradient_against_differences():
    """A directional difference of the oracle's forward at the kernel's fp32
    inputs: the step 1e-4 leaves about 1e-8 relative, the kernel 1e-6."""
    x, dy, w, b = make(6, 200, torch.float32, torch.float32, seed=10)
    y, mean, rstd = api.layer_norm_fwd(x, w, b)
    grads = [host(t) for t in api.layer_norm_bwd(dy, x, mean, rstd, w, b)]
    args = [host(x), host(w), host(b)]
    r = np.random.default_rng(0)
    for i, g in enumerate(grads):
        d = r.standard_normal(args[i].shape)
        v = []
        for h in (1e-4, -1e-4):
            a = list(args)
            a[i] = a[i] + h * d
            v.append((ops.layer_norm(*a)[0] * host(dy)).sum())
        num, ana = (v[0] - v[1]) / 2e-4, (g * d).sum()
        assert abs(num - ana) <= 1e-5 * np.linalg.norm(g) * np.linalg.norm(d)


def test_statistics_of_a_bad_row():
    """The saved statistics say so too: a NaN is no rstd of 1 / sqrt(eps)."""
    for C in (100, 20000):
        x = torch.randn(3, C, device="cuda")
        x[1, 5] = float("nan")
        _, mean, rstd = api.layer_norm_fwd(x)
        torch.cuda.synchronize()
        assert torch.isfinite(rstd[[0, 2]]).all() and rstd[1].isnan() and mean[1].isnan()
