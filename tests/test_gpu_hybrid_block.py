"""The operators together, as a hybrid block uses them: layer norm, the block's
projections, rotary positions, softmax attention (or the frame scan) and the
output projection, against the same chain of fp64 oracles; frames streamed
against a key cache; and a training step's gradients.

Tolerance.  Each stage rounds its result to bf16 once, 2^-9 / sqrt(3) = 1.1e-3
rms relative for values spread over a binade, at most 1.7e-3; the chain has
seven such stages (norm, projection, rotation, probabilities, attention output,
output projection, and the scores' own error of about two roundings of q and k),
which add to at most 7 x 1.7e-3 = 1.2e-2 in relative Frobenius norm.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import block as oblock, ops
from gated_deltanet_scan_amd import api, autograd, inputs

pytestmark = pytest.mark.gpu

BAR = 1.2e-2
AXES = (16, 24, 24)


def host(t):
    return t.detach().double().cpu().numpy()


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16).contiguous()


def rel(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


def setup(F=3, Hg=5, Wg=9, C=256, H=4, D=64, seed=3):
    w = inputs.make_block(1, F, Hg * Wg, C, H, D, seed=seed)
    g = np.random.default_rng(seed)
    return w, inputs.round_bf16(1 + 0.2 * g.standard_normal(C).astype(np.float32)), \
        inputs.round_bf16(0.2 * g.standard_normal(C).astype(np.float32)), api.video_positions(F, Hg, Wg)


def in_half(w, nw, nb, pos):
    """Norm, projections and rotation on the GPU: (q, k, v, beta, alpha) with q
    and k before and after the rotation."""
    x, _, _ = api.layer_norm_fwd(bf(w.x), bf(nw), bf(nb), return_stats=False)
    q, k, v, bl, al = api.block_in_proj(x, bf(w.w_qkv), bf(w.w_gate), H=w.H, D=w.D)
    q, k = api.rotary(q, k, pos, axes=AXES)
    return q, k, v, bl, al


def in_half_ref(w, nw, nb, pos):
    x = ops.layer_norm(w.x, nw, nb)[0]
    q, k, v, bl, al = oblock.block_in_proj(x, w.w_qkv, w.w_gate)
    T = w.F * w.N
    p = host(pos).reshape(T, 3)
    q, k = (ops.rotary(t.reshape(T, w.H, w.D), p, AXES).reshape(t.shape) for t in (q, k))
    return q, k, v, bl, al


def test_softmax_block():
    w, nw, nb, pos = setup()
    q, k, v, _, _ = in_half(w, nw, nb, pos)
    o, _ = api.attention_fwd(q, k, v, causal=True)
    y = api.block_out_proj(o, bf(w.w_out))
    torch.cuda.synchronize()
    rq, rk, rv, _, _ = in_half_ref(w, nw, nb, pos)
    T = w.F * w.N
    ro, _ = ops.attention(*[t.reshape(T, w.H, w.D) for t in (rq, rk, rv)], causal=True, block=w.N)
    ry = oblock.block_out_proj(ro.reshape(1, w.F, w.N, w.H, w.D), w.w_out)
    e = rel(host(y), ry)
    print("softmax block: rel %.2e" % e)
    assert e <= BAR


def test_scan_block_with_rotated_keys():
    w, nw, nb, pos = setup(seed=4)
    q, k, v, bl, al = in_half(w, nw, nb, pos)
    o, _ = api.frame_scan_fwd(q, k, v, bl, al, None, gates_are_logits=True)
    y = api.block_out_proj(o, bf(w.w_out))
    torch.cuda.synchronize()
    ro, _ = oracle.scan(*in_half_ref(w, nw, nb, pos), None, gates_are_logits=True)
    e = rel(host(y), oblock.block_out_proj(ro, w.w_out))
    print("scan block: rel %.2e" % e)
    assert e <= BAR


def test_streamed_frames_equal_the_clip():
    """Frame by frame against a cache with room: positions from the frame's
    offset, keys written behind those so far, k_len on the device.  The same
    products in another split of the keys: equal to rounding, 2 x 2^-8."""
    w, nw, nb, pos = setup(F=5)
    q, k, v, _, _ = in_half(w, nw, nb, pos)
    clip, _ = api.attention_fwd(q, k, v, causal=True)
    room = 7 * w.N
    kc, vc = (torch.full((1, room, w.H, w.D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x, _, _ = api.layer_norm_fwd(bf(w.x), bf(nw), bf(nb), return_stats=False)
    for f in range(w.F):
        qf, kf, vf, _, _ = api.block_in_proj(x[:, f:f + 1].contiguous(), bf(w.w_qkv), bf(w.w_gate), H=w.H, D=w.D)
        pf = api.video_positions(1, 5, 9, frame_offset=f)
        qf, kf = api.rotary(qf, kf, pf, axes=AXES)
        kc[:, f * w.N:(f + 1) * w.N], vc[:, f * w.N:(f + 1) * w.N] = kf[:, 0], vf[:, 0]
        n = torch.tensor([(f + 1) * w.N], dtype=torch.int32, device="cuda")
        of, _ = api.attention_fwd(qf[:, 0], kc, vc, causal=True, causal_block=w.N, k_len=n)
        torch.cuda.synchronize()
        assert torch.equal(qf, q[:, f:f + 1]) and torch.equal(kf, k[:, f:f + 1])
        d = (of.float() - clip[:, f].float()).abs()
        assert (d <= 2 * 2.0 ** -8 * clip[:, f].float().abs() + 2e-3 * clip.float().abs().max()).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_training_step_gradients(dtype):
    """norm -> q, k, v projections (torch products) -> rotary -> attention over
    two packed sequences, the gradients of every parameter against 64-bit
    autograd of the plain formulas."""
    g = torch.Generator().manual_seed(5)
    T, C, Hq, Hk, D = 100, 96, 4, 2, 32
    lens, block, axes = [60, 40], 20, (8, 12, 12)
    mk = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(dtype)
    x, w, b = mk(T, C), 1 + mk(C, std=0.2), mk(C, std=0.2)
    wq, wk, wv = mk(Hq * D, C, std=C ** -0.5), mk(Hk * D, C, std=C ** -0.5), mk(Hk * D, C, std=C ** -0.5)
    do = mk(T, Hq, D)
    pos = torch.randint(0, 30, (T, 3), generator=g, dtype=torch.int32)
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, b, wq, wk, wv)]
    lx, lw, lb, lq, lk, lv = leaves
    h = autograd.layer_norm(lx, lw, lb)
    q, k, v = ((h @ m.t()).reshape(T, -1, D) for m in (lq, lk, lv))
    q, k = autograd.rotary(q, k, pos.cuda(), axes=axes)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    o = autograd.attention(q, k, v, causal=True, causal_block=block, cu_q=cu, max_q=60, max_k=60)
    o.backward(do.cuda())
    torch.cuda.synchronize()

    ref = [t.double().requires_grad_(True) for t in (x, w, b, wq, wk, wv)]
    rx, rw, rb, rq, rk, rv = ref
    m = rx.mean(-1, keepdim=True)
    h = (rx - m) / ((rx - m) ** 2).mean(-1, keepdim=True).add(1e-6).sqrt() * rw + rb
    q, k, v = ((h @ t.t()).reshape(T, -1, D) for t in (rq, rk, rv))
    ang = torch.cat([pos[:, a:a + 1].double() * 10000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d)
                     for a, d in enumerate(axes)], -1)[:, None]

    def turn(t):
        z = torch.view_as_complex(t.reshape(T, -1, D // 2, 2).contiguous()) * torch.polar(torch.ones_like(ang), ang)
        return torch.view_as_real(z).reshape(T, -1, D)

    q, k = turn(q), turn(k)
    at, outs = 0, []
    for n in lens:
        sl = slice(at, at + n)
        kk, vv = (t[sl].repeat_interleave(Hq // Hk, 1).transpose(0, 1) for t in (k, v))
        s = q[sl].transpose(0, 1) @ kk.transpose(1, 2) * D ** -0.5
        p = torch.arange(n)
        s = s.masked_fill(~(p[None] // block <= p[:, None] // block), float("-inf")).softmax(-1)
        outs.append((s @ vv).transpose(0, 1))
        at += n
    ro = torch.cat(outs)
    ro.backward(do.double())
    # fp32: sums of at most 100 terms and five products in a row, 5 x 100 x 2^-24 = 3e-5 at the very most
    bar = 3e-5 if dtype == torch.float32 else 2 * BAR             # bf16: forward and backward stages
    for n, a, r in zip(("o", "x", "w", "b", "wq", "wk", "wv"), [o] + [t.grad for t in leaves],
                       [ro] + [t.grad for t in ref]):
        e = rel(host(a), r.detach().numpy())
        print("%s: rel %.2e" % (n, e))
        assert e <= bar, n


def test_second_derivatives_are_refused():
    x = torch.randn(4, 96, device="cuda", requires_grad=True)
    q = torch.randn(1, 4, 2, 32, device="cuda", requires_grad=True)
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    for leaf, y in ((x, autograd.layer_norm(x)), (q, autograd.rotary(q, None, pos, axes=(32,))[0]),
                    (q, autograd.attention(q, q, q))):
        g, = torch.autograd.grad((y * y).sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.sum().backward()
