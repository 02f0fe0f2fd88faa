"""Softmax attention on views of one token per sequence that lie far apart: the
first token of a batched cache's slots, the last token of long sequences.  The
kernels read the same values as from packed copies, so the results are the same
bit for bit; where one key is visible, o is that key's v up to rounding.  And
bounds of the lengths far above them.
"""
import ctypes

import pytest
import torch

from gated_deltanet_scan_amd import _lib, api, autograd

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype,Hq,Hk,D", [(BF, 16, 8, 128), (BF, 8, 8, 64), (BF, 16, 4, 32), (BF, 8, 4, 16),
                                           (F32, 8, 2, 64)])
@pytest.mark.parametrize("lq,lk", [(1, 1), (1, 3), (3, 1)])
def test_far_single_tokens(dtype, Hq, Hk, D, lq, lk):
    room = (1 << 20) // (Hk * D) + 3                      # a token stride past 2^20
    x, kc, vc = rand((2, room, Hq, D), dtype, 1), rand((2, room, Hk, D), dtype, 2), rand((2, room, Hk, D), dtype, 3)
    q = x[:, -1:] if lq == 1 else x[:, -lq:].contiguous()
    k, v = kc[:, :lk], vc[:, :lk]
    args = [t.contiguous() for t in (q, k, v)]
    o, lse = api.attention_fwd(q, k, v, causal=lq <= lk)
    o2, lse2 = api.attention_fwd(*args, causal=lq <= lk)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if lk == 1:
        # o = fl(fl(p v) fl(1 / p)) with p next to 1: three roundings, 3 2^-24 (1 + 2^-23)^2 < 4 2^-24
        # in fp32; in bf16 p rounds to 1 and what l is off by, below 2^-20, does not move v's rounding
        want = v.repeat_interleave(Hq // Hk, dim=2).expand_as(o).double()
        assert torch.all((o.double() - want).abs() <= (0 if dtype == BF else 4 * 2.0 ** -24) * want.abs())
    do = rand(o.shape, dtype, 4)
    for a, b in zip(api.attention_bwd(q, k, v, o, lse, do, causal=lq <= lk),
                    api.attention_bwd(*args, o, lse, do, causal=lq <= lk)):
        assert torch.equal(a, b)
    leaves = [t.detach().clone().requires_grad_() for t in (x, kc, vc)]
    y = autograd.attention(leaves[0][:, -lq:] if lq == 1 else leaves[0][:, -lq:].contiguous(), leaves[1][:, :lk],
                           leaves[2][:, :lk], causal=lq <= lk)
    y.backward(do)
    packed = api.attention_bwd(*args, o, lse, do, causal=lq <= lk)
    for leaf, g, at in zip(leaves, packed, (slice(room - lq, room), slice(0, lk), slice(0, lk))):
        assert torch.equal(leaf.grad[:, at], g)
        assert leaf.grad.count_nonzero() == g.count_nonzero()         # and zeros elsewhere


def test_rollout_from_its_first_token():
    """k[:, :n] of a long cache from n = 1 on, as a batched rollout reads it."""
    x, kc, vc = rand((2, 32768, 8, 128), BF, 5), rand((2, 32768, 8, 128), BF, 6), rand((2, 32768, 8, 128), BF, 7)
    for n in (1, 2, 3, 65):
        q = x[:, n - 1:n]
        o, lse = api.attention_fwd(q, kc[:, :n], vc[:, :n], causal=True)
        k_len = torch.full((2,), n, dtype=torch.int32, device="cuda")
        o2, lse2 = api.attention_fwd(q.contiguous(), kc[:, :66], vc[:, :66], causal=True, k_len=k_len)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), n


@pytest.mark.parametrize("dtype,Hq,Hk,D,lens_q,lens_k", [
    (BF, 8, 1, 128, (1, 1), (5000, 12000)), (F32, 6, 2, 64, (70, 1, 0), (300, 400, 5)), (BF, 4, 2, 32, (900,), (1300,))])
def test_bounds_far_above_the_lengths(dtype, Hq, Hk, D, lens_q, lens_k):
    """max_q = 2^30 / Hq and max_k = 2^30 are bounds like any other."""
    lib, n = _lib.load(), len(lens_q)
    cu_q, cu_k = [torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).int().cuda() for lens in (lens_q, lens_k)]
    tq, tk = sum(lens_q), sum(lens_k)
    q, k, v, do = rand((tq, Hq, D), dtype, 1), rand((tk, Hk, D), dtype, 2), rand((tk, Hk, D), dtype, 3), \
        rand((tq, Hq, D), dtype, 4)
    o, lse = api.attention_fwd(q, k, v, cu_q=cu_q, cu_k=cu_k, causal=True)
    ref = [o, lse, *api.attention_bwd(q, k, v, o, lse, do, cu_q=cu_q, cu_k=cu_k, causal=True)]
    got = [torch.full_like(t, float("nan")) for t in ref]
    d = ctypes.byref(_lib.GdnAttnDesc(tq, tk, 0, 0, 0, 0, n, Hq, Hk, D, (1 << 30) // Hq, 1 << 30, 1,
                                      _lib.GDN_BF16 if dtype == BF else _lib.GDN_F32, _lib.GDN_FLAG_ATTN_CAUSAL,
                                      D ** -0.5))
    size = max(lib.gdn_attn_workspace_size(d), lib.gdn_attn_workspace_size_bwd(d))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    P = [t.data_ptr() for t in (q, k, v, do, cu_q, cu_k, ws, *got)]
    assert lib.gdn_attn_fwd(d, *P[:3], P[4], P[5], None, P[7], P[8], P[6], size, stream) == 0
    assert lib.gdn_attn_bwd(d, *P[:3], P[7], P[8], P[3], P[4], P[5], *P[9:12], P[6], size, stream) == 0
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
