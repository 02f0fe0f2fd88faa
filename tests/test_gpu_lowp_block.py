"""The low-precision operators together, as a softmax block of a hybrid backbone
serves with them: norm with an 8-bit output, 8-bit projections, rotary positions, a
block-scaled cache written frame by frame (and token by token), attention over it, and
the 8-bit output projection.

Tolerance.  The same chain in float64 over the same codes: every stage's own input is
taken from the GPU, so a stage's error is its own rounding.
"""
import os

import numpy as np
import pytest
import torch

from gated_deltanet_scan_amd import api, inputs
from oracle import ops
from test_gpu_attention import check, dense

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
C, H, D, N = 256, 4, 64, 45
AXES = (16, 24, 24)


def host(t):
    return t.detach().double().cpu().numpy()


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn((3 * H * D, C), generator=g) * C ** -0.5
    wo = torch.randn((C, H * D), generator=g) * (H * D) ** -0.5
    return inputs.to_fp8_weight(w.cuda()), inputs.to_fp8_weight(wo.cuda()), (1 + 0.2 * torch.randn(C, generator=g)).to(BF).cuda()


def block(x, res, at, cache, w, wo, nw, n_len, fp4, frame):
    """One step of the block: x [B, n, C] onto a cache in use up to n_len with the new tokens."""
    B, n, _ = x.shape
    h, hs, total = api.rms_norm_fwd_fp8(x, nw, res)
    q, k, v = api.matmul_fp8(h, hs, *w, parts=3).view(3, B, n, H, D)
    q, k = api.rotary(q, k, at, axes=AXES)
    api.cache_write(k, v, *cache, k_len=n_len)
    fwd = api.attention_fwd_fp4 if fp4 else api.attention_fwd_fp8
    o, lse = fwd(q, *cache, causal=True, causal_block=frame, k_len=n_len)
    os, oss = api.quantize_fp8(o.view(B, n, H * D))
    return api.matmul_fp8(os, oss, *wo), total, (q, k, v, o, lse, h, hs, os, oss)


@pytest.mark.parametrize("fp4", [True, False], ids=["fp4", "fp8"])
def test_streamed_frames(fp4):
    """Frames streamed into a cache, each stage against its formula on what the stage before gave."""
    B, F = 2, 3
    w, wo, nw = weights()
    cache = api.cache_empty(B, F * N + 7, H=H, D=D, fp4=fp4)
    g = torch.Generator().manual_seed(1)
    kept = []
    for f in range(F):
        x, res = (torch.randn((B, N, C), generator=g).to(BF).cuda() for _ in range(2))
        at = api.video_positions(1, 5, 9, frame_offset=f).view(N, 3)
        n_len = torch.full((B,), (f + 1) * N, dtype=torch.int32, device="cuda")
        y, total, (q, k, v, o, lse, h, hs, os, oss) = block(x, res, at, cache, w, wo, nw, n_len, fp4, N)
        assert torch.equal(total, (x.float() + res.float()).to(BF))
        kept.append((k, v))
        # the cache holds every frame's encoding
        kr, vr = api.cache_read(*cache, dtype=torch.float32, k_len=n_len)
        enc = inputs.to_mxfp4 if fp4 else inputs.to_mxfp8
        for i, t in enumerate((kr, vr)):
            for j, kv in enumerate(kept):
                want = enc(kv[i].float().cpu().numpy())[2]
                assert np.array_equal(t[:, j * N:(j + 1) * N].cpu().numpy(), want)
        for b in range(B):
            xq = host(q[b])
            m = (f + 1) * N
            val, bar = dense(xq, host(kr[b, :m]), host(vr[b, :m]), np.zeros_like(xq), True, N, D ** -0.5, BF)
            check(host(o[b]), val["o"], bar["o"], "o")
            check(host(lse[b]), val["lse"], bar["lse"], "lse")
        # both projections, relative to their norms: bf16's rounding
        ref = ops.matmul(host(h).reshape(-1, C), host(hs).reshape(-1, C // 128), *(host(t) for t in w))
        got = host(v).reshape(B * N, H * D)
        ref = ref[:, 2 * H * D:]
        assert np.linalg.norm(got - ref) <= 2.0 ** -8 / 3 ** 0.5 * np.linalg.norm(ref)
        ref = ops.matmul(host(os).reshape(-1, H * D), host(oss).reshape(-1, H * D // 128), *(host(t) for t in wo))
        assert np.linalg.norm(host(y).reshape(ref.shape) - ref) <= 2.0 ** -8 / 3 ** 0.5 * np.linalg.norm(ref)


@pytest.mark.parametrize("fp4", [True, False], ids=["fp4", "fp8"])
def test_tokens_captured_and_replayed(fp4):
    """Single tokens, the step captured once and replayed as the lengths on the device grow: every replay gives what
    eager calls give."""
    B, room, first = 3, 200, [5, 63, 128]
    w, wo, nw = weights(2)
    g = torch.Generator().manual_seed(3)
    steps = [[torch.randn((B, 1, C), generator=g).to(BF).cuda() for _ in range(2)] for _ in range(5)]
    old = [torch.randn((B, room, H, D), generator=g).to(BF).cuda() for _ in range(2)]

    def start():
        cache = api.cache_empty(B, room, H=H, D=D, fp4=fp4)
        n = torch.tensor(first, dtype=torch.int32, device="cuda")
        for b in range(B):
            api.cache_write(old[0][b:b + 1, :first[b]], old[1][b:b + 1, :first[b]],
                            *[t[b:b + 1, :first[b]] for t in cache])
        return cache, n, torch.zeros((B, 1, 3), dtype=torch.int32, device="cuda")

    cache, n, pos = start()
    ref = []
    for x, r in steps:
        n += 1
        pos[:, 0, 0] = n
        y, total, more = block(x, r, pos, cache, w, wo, nw, n, fp4, 1)
        ref.append((y.clone(), total.clone(), more[4].clone()))
    torch.cuda.synchronize()
    want = [t.clone() for t in cache]

    cache, n, pos = start()
    x, r = (torch.zeros_like(t) for t in steps[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, total, more = block(x, r, pos, cache, w, wo, nw, n, fp4, 1)
    for i, (a, b) in enumerate(steps):
        x.copy_(a)
        r.copy_(b)
        n += 1
        pos[:, 0, 0] = n
        graph.replay()
        torch.cuda.synchronize()
        for got, e in zip((y, total, more[4]), ref[i]):
            assert torch.equal(got, e), i
    for a, b in zip(cache, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_the_documented_block():
    """README's low-precision block as it stands, three frames: what the cache holds, the attention over all of it,
    and the output projection (an identity here)."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code = [line[4:] for line in text[text.index("    cache = api.cache_empty"):].split("\nA frame of")[0].splitlines()]
    once, each = "\n".join(code[:code.index("")]), "\n".join(code[code.index(""):])
    B, N, W, F = 2, 880, 2048, 3
    g = torch.Generator().manual_seed(5)
    w = torch.randn((3 * W, W), generator=g) * W ** -0.5
    (w_qkv, w_qkv_s), (w_out, w_out_s) = inputs.to_fp8_weight(w.cuda()), inputs.to_fp8_weight(torch.eye(W).cuda())
    names = dict(api=api, B=B, N=N, room=F * N + 5, w_qkv=w_qkv, w_qkv_s=w_qkv_s, w_out=w_out, w_out_s=w_out_s,
                 w_norm=torch.ones(W, device="cuda"), y=torch.randn((B, N, W), generator=g).to(BF).cuda(),
                 x=torch.zeros((B, N, W), dtype=BF, device="cuda"))
    exec(once, names)
    for f in range(F):
        names.update(f=f, n=torch.full((B,), (f + 1) * N, dtype=torch.int32, device="cuda"))
        exec(each, names)
        k, v = (t[:, :(f + 1) * N] for t in api.cache_read(*names["cache"], dtype=torch.float32, k_len=names["n"]))
        want = inputs.to_mxfp4(names["k"].float().cpu().numpy())[2]
        assert np.array_equal(k[:, f * N:].cpu().numpy(), want)
        ref, _ = api.attention_fwd(names["q"], k.to(BF), v.to(BF), causal=True, causal_block=N)
        o = names["o"]
        assert (o.double() - ref.double()).norm() <= 2 * 2.5e-3 * ref.double().norm()      # each is 2.5e-3 from 64 bits
        y = names["y"]
        # the output projection is the identity: what is left is the 8-bit rounding of o (half a step of 2^-3, and a
        # group's smallest values to 2^-10 of its largest)
        assert y.shape == (B, N, W) and names["x"].shape == (B, N, W)
        og = o.flatten(-2).float()
        top = og.abs().unflatten(-1, (-1, 128)).amax(-1, keepdim=True).expand(-1, -1, -1, 128).flatten(-2)
        assert torch.all((y.float() - og).abs() <= (2.0 ** -4 + 2.0 ** -8) * 1.01 * og.abs() + 2.0 ** -18 * 1.01 * top)
