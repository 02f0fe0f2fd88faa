"""Rotary positions on the GPU (gdn_rotary) against the fp64 oracle
(oracle/ops.py).

Tolerance.  u = 2^-24.  The angle is reduced to [-1/2, 1/2] turns in 64 bits
and rounded once to fp32 (2^-26 turns at most, 2 pi 2^-26 = 1.6 u radians),
fp32's sine and cosine add at most 2 u, each product and the sum u of its
size: with m = |x| + |y| of the pair, every output is within 8 u m, plus half
a step of the output type (2^-8 relative for bf16, u for fp32).  The 64-bit
angle itself, about position * 2^-53, is far below that for the positions here.
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


def check(got, x, pos, axes, dtype, name, **kw):
    T_, H, D = x.shape
    ref = ops.rotary(x, pos, axes, **kw)
    R = sum(axes)
    m = np.zeros_like(ref)
    a = np.abs(x)
    if kw.get("halves"):
        s = a[..., :R // 2] + a[..., R // 2:R]
        m[..., :R // 2], m[..., R // 2:R] = s, s
    else:
        s = a[..., 0:R:2] + a[..., 1:R:2]
        m[..., 0:R:2], m[..., 1:R:2] = s, s
    bar = 8 * U * m + T[dtype] * np.abs(ref)
    err = np.abs(got - ref)
    assert np.all(err <= bar), (name, (err - bar).max())
    assert np.array_equal(got[..., R:], x[..., R:]), name


CASES = [
    # tokens, pos rows, Hq, Hk, D, axes
    (1, 1, 1, 1, 8, (8,)),
    (1, 1, 1, 0, 256, (100, 100, 56)),
    (7, 7, 3, 1, 16, (4, 6, 6)),
    (100, 50, 16, 16, 128, (44, 42, 42)),
    (333, 333, 5, 2, 64, (20, 20, 22)),
    (61, 61, 12, 4, 64, (16, 16, 16)),
    (40, 20, 1, 7, 40, (10, 10)),
    (29, 29, 2, 2, 32, (10, 0, 4, 16)),
    (5000, 1250, 4, 1, 32, (8, 8, 8)),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("halves", [False, True], ids=["pairs", "halves"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%dP%dHq%dHk%dD%d" % c[:5])
def test_against_the_oracle(case, halves, dtype):
    tokens, rows, Hq, Hk, D, axes = case
    g = torch.Generator().manual_seed(tokens + D)
    q, k = torch.randn((tokens, Hq, D), generator=g), torch.randn((tokens, Hk, D), generator=g)
    pos = torch.randint(0, 200000, (rows, len(axes)), generator=g, dtype=torch.int32)
    q, k, pos = q.to(dtype).cuda(), k.to(dtype).cuda(), pos.cuda()
    # token t takes row t % rows: give the token axes as [batch, rows]
    shape = lambda t: t.reshape(tokens // rows, rows, *t.shape[1:])
    for inverse in (False, True):
        qo, ko = api.rotary(shape(q), shape(k) if Hk else None, pos, axes=axes, halves=halves, inverse=inverse)
        torch.cuda.synchronize()
        check(host(qo).reshape(q.shape), host(q), host(pos), axes, dtype, "q", halves=halves, inverse=inverse)
        if Hk:
            check(host(ko).reshape(k.shape), host(k), host(pos), axes, dtype, "k", halves=halves, inverse=inverse)


@pytest.mark.parametrize("halves", [False, True], ids=["pairs", "halves"])
def test_in_place_equals_out_of_place(halves):
    q, k = (torch.randn((2, 300, h, 128), device="cuda").bfloat16() for h in (16, 4))
    pos = torch.randint(0, 900, (300, 3), dtype=torch.int32, device="cuda")
    kw = dict(axes=(40, 40, 40), halves=halves)
    qo, ko = api.rotary(q, k, pos, **kw)
    q2, k2 = q.clone(), k.clone()
    api.rotary(q2, k2, pos, q_out=q2, k_out=k2, **kw)
    torch.cuda.synchronize()
    assert torch.equal(qo, q2) and torch.equal(ko, k2)


def test_float_positions_and_nonfinite_passthrough():
    """Fractional and negative positions; features past the axes keep their
    bits, infinities included."""
    q = torch.randn((50, 2, 32), device="cuda")
    q[3, 1, 30], q[4, 0, 31] = float("inf"), float("nan")
    pos = torch.randn((50, 2), device="cuda") * 100
    qo, none = api.rotary(q, None, pos, axes=(10, 16), theta=500.0)
    torch.cuda.synchronize()
    assert none is None
    assert torch.equal(qo[..., 26:].view(torch.int32), q[..., 26:].view(torch.int32))
    x = host(q)[..., :26]
    check(host(qo)[..., :26], x, host(pos), (10, 16), torch.float32, "q", theta=500.0)


def test_video_positions():
    pos = api.video_positions(3, 4, 5, frame_offset=7)
    assert pos.shape == (3, 20, 3) and pos.dtype == torch.int32
    assert pos[2, 13].tolist() == [9, 2, 3]


def test_empty():
    q = torch.empty((0, 4, 64), device="cuda", dtype=torch.bfloat16)
    pos = torch.empty((0, 2), device="cuda", dtype=torch.int32)
    qo, _ = api.rotary(q, None, pos, axes=(32, 32))
    assert qo.shape == q.shape


def test_autograd_and_differences():
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn((2, 9, h, 16), generator=g).cuda().requires_grad_(True) for h in (4, 2))
    pos = torch.randint(0, 50, (9, 2), generator=g, dtype=torch.int32).cuda()
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    qo, ko = autograd.rotary(q, k, pos, axes=(8, 6), halves=True)
    ((qo * dq).sum() + (ko * dk).sum()).backward()
    rq, rk = api.rotary(dq, dk, pos, axes=(8, 6), halves=True, inverse=True)
    torch.cuda.synchronize()
    assert torch.equal(q.grad, rq) and torch.equal(k.grad, rk)
    d = np.random.default_rng(0).standard_normal((18, 4, 16))
    x, go = host(q).reshape(18, 4, 16), host(dq).reshape(18, 4, 16)
    v = [(ops.rotary(x + h * d, host(pos), (8, 6), halves=True) * go).sum() for h in (1e-4, -1e-4)]
    ana = (host(q.grad).reshape(18, 4, 16) * d).sum()
    assert abs((v[0] - v[1]) / 2e-4 - ana) <= 1e-5 * np.linalg.norm(go) * np.linalg.norm(d)
    # queries alone, and a gradient for the keys only
    q2 = q.detach().clone().requires_grad_(True)
    autograd.rotary(q2, None, pos, axes=(8, 6))[0].sum().backward()
    k2 = k.detach().clone().requires_grad_(True)
    autograd.rotary(q.detach(), k2, pos, axes=(8, 6))[1].sum().backward()
    torch.cuda.synchronize()
    assert torch.isfinite(q2.grad).all() and torch.isfinite(k2.grad).all()


def test_graph_replays():
    q, k = (torch.randn((2, 880, h, 128), device="cuda").bfloat16() for h in (16, 16))
    pos = api.video_positions(1, 22, 40).reshape(880, 3)
    kw = dict(axes=(44, 42, 42))
    qr, kr = api.rotary(q, k, pos, **kw)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.rotary(q, k, pos, q_out=qo, k_out=ko, **kw)
    for _ in range(3):
        qo.zero_()
        ko.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, qr) and torch.equal(ko, kr)
