"""The low-precision operators past 2^32 elements, over thousands of sequences, and over no keys at all."""
import numpy as np
import pytest
import torch

from gated_deltanet_scan_amd import api, inputs
from test_gpu_attention import BF, starts
from test_gpu_attention_mx import FORMATS, compare, encode, fwd, rand

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def raw(t):
    return t.view(torch.uint8)


@FORMATS
def test_long_cache(fp4):
    """A cache of more than 2^32 bytes: tokens written at its end, attention over the end alone and over all of it,
    and the end read back.

    All keys but the last 300 are zeros with values of zero, so p is 1 there and
    o = sum over the 300 of e^s v / (T - 300 + sum e^s).  With v > 0 nothing cancels: p
    and o round to bf16 (2^-8 each), the rest is fp32 with fewer than 2^12 additions that
    round in a row (sums of ones are exact): 2^-7 + 2^-12 relative, and 2^-12 for the sum.
    """
    H, D, n = 8, 128, 300
    T = 2 ** 32 // (H * D // 2 if fp4 else H * D) + 777
    cache = api.cache_empty(T, H=H, D=D, fp4=fp4)
    k, v = rand((n, H, D), 1), rand((n, H, D), 2).abs() + 0.5
    k, v = k.to(BF), v.to(BF)
    (kc, ks, kv), (vc, vs, vv) = encode(k.float(), fp4), encode(v.float(), fp4)
    api.cache_write(k.cuda(), v.cuda(), *cache, cu_new=dev([0, n]), cu_k=dev([0, T]))
    for got, want in zip(cache, (kc, ks, vc, vs)):
        assert torch.equal(raw(got[T - n:]), raw(want))
        assert not raw(got[T - n - 2000:T - n]).any() and not raw(got[:2000]).any()
    for lq in (1, 20, 40):
        q = rand((lq, H, D), lq).to(BF).cuda()
        o, lse = fwd(fp4)(q, *cache, cu_q=dev([0, lq]), cu_k=dev([T - n, T]), max_k=n)
        compare(q, kv, vv, [0], [0], [lq], [n], False, 1, D ** -0.5, o, lse)
        o, lse = fwd(fp4)(q, *cache, cu_q=dev([0, lq]), cu_k=dev([0, T]))
        e = np.exp(np.einsum("qhd,khd->qhk", q.double().cpu().numpy(), kv) * D ** -0.5)
        total = T - n + e.sum(-1)
        ref = np.einsum("qhk,khd->qhd", e, vv) / total[..., None]
        err = np.abs(o.double().cpu().numpy() / ref - 1).max()
        print("lq %d: %.2e of %.2e" % (lq, err, 2.0 ** -7 + 2.0 ** -12))
        assert err <= 2.0 ** -7 + 2.0 ** -12
        assert np.abs(lse.double().cpu().numpy() - np.log(total)).max() <= 2.0 ** -12
    kr, vr = api.cache_read(*cache, cu_k=dev([T - n, T]))
    assert np.array_equal(kr[T - n:].double().cpu().numpy(), kv) and np.array_equal(vr[T - n:].double().cpu().numpy(), vv)


def test_long_activations():
    """More than 2^32 values: the last rows as they come alone."""
    rows, C, n = 2 ** 21 + 101, 2048, 5000
    w = (1 + rand((C,), 1, 0.2)).to(BF).cuda()
    x = torch.zeros((rows, C), dtype=BF, device="cuda")
    r = torch.zeros_like(x)
    x[-n:], r[-n:] = rand((n, C), 2).to(BF).cuda(), rand((n, C), 3).to(BF).cuda()
    for got, want in ((api.rms_norm_fwd_fp8(x, w, r), api.rms_norm_fwd_fp8(x[-n:], w, r[-n:])),
                      (api.quantize_fp8(x), api.quantize_fp8(x[-n:]))):
        for a, b in zip(got, want):
            assert torch.equal(raw(a[-n:]), raw(b))
        assert not raw(got[0][:-n]).any()


@pytest.mark.parametrize("M,N,K", [(2 ** 22 + 77, 96, 1040), (2 ** 21 + 33, 2304, 128)])
def test_long_products(M, N, K):
    """x or y of more than 2^32 values: the last rows against 64 bits, within the bar of a product."""
    n = 500
    x = torch.zeros((M, K), dtype=torch.float8_e4m3fn, device="cuda")
    xs = torch.zeros((M, -(-K // 128)), device="cuda")
    x[-n:], xs[-n:] = api.quantize_fp8(rand((n, K), 1).cuda())
    w, ws = inputs.to_fp8_weight(rand((N, K), 2).cuda())
    y = api.matmul_fp8(x, xs, w, ws)
    xv = x[-n:].double() * xs[-n:].double().repeat_interleave(128, 1)[:, :K]
    wv = w.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    ref, size = xv @ wv.t(), xv.abs() @ wv.abs().t()
    err = (y[-n:].double() - ref).abs()
    assert torch.all(err <= 7 * 2.0 ** -13 * size + (24 + K // 128) * 2.0 ** -24 * size + 2.0 ** -8 * ref.abs())
    assert not y[:1000].any() and not y[-n - 1000:-n].any()


@FORMATS
@pytest.mark.parametrize("most", [2, 150])
def test_thousands_of_sequences(most, fp4):
    """Ragged requests by the thousand, in the kernel for few rows and (two sequences of 150 queries) in the tiles."""
    n = 3000
    r = np.random.default_rng(7)
    lens_q, lens_k = r.choice([0, 1, 1, 2], n), r.choice([0, 1, 5, 40, 70], n)
    lens_q[[0, 777]] = most
    lens_k[[0, 1500]] = 900
    cu_q, cu_k = starts(lens_q), starts(lens_k)
    q = rand((int(cu_q[-1]), 4, 32), n).to(BF).cuda()
    kc, ks, kv = encode(rand((int(cu_k[-1]), 2, 32), n + 1), fp4)
    vc, vs, vv = encode(rand((int(cu_k[-1]), 2, 32), n + 2), fp4)
    o, lse = fwd(fp4)(q, kc, ks, vc, vs, causal=True, cu_q=torch.from_numpy(cu_q).cuda(),
                      cu_k=torch.from_numpy(cu_k).cuda(), max_q=most)
    torch.cuda.synchronize()
    compare(q, kv, vv, cu_q, cu_k, lens_q, lens_k, True, 1, 32 ** -0.5, o, lse)


@FORMATS
@pytest.mark.parametrize("lq", [1, 50])
def test_no_keys(lq, fp4):
    """Caches without a place, and empty batches: rows of zeros with a sum's logarithm of -inf."""
    cache = api.cache_empty(2, 0, H=2, D=64, fp4=fp4)
    q = rand((2, lq, 4, 64), 1).to(BF).cuda()
    o, lse = fwd(fp4)(q, *cache, causal=True)
    assert not o.any() and torch.all(lse == -float("inf"))
    api.cache_write(q[:, :, :2], q[:, :, :2], *cache)
    assert api.cache_read(*cache)[0].shape == (2, 0, 2, 64)
    o, lse = fwd(fp4)(q[:0], *[t[:0] for t in api.cache_empty(2, 3, H=2, D=64, fp4=fp4)])
    assert o.shape == (0, lq, 4, 64)
    o, lse = fwd(fp4)(q[:, :0], *api.cache_empty(2, 3, H=2, D=64, fp4=fp4))
    assert o.shape == (2, 0, 4, 64)


@FORMATS
def test_more_rows_than_a_join_takes(fp4):
    """70000 requests with room for 32 queries each, on 8 heads: more (row, head) places than one launch of the join
    may have, which short keys do not need."""
    n, H, D, most = 70000, 8, 32, 32
    r = np.random.default_rng(9)
    lens_q, lens_k = (r.random(n) < 0.01).astype(np.int64), r.choice([0, 0, 0, 0, 1, 3], n)
    lens_q[[5, n - 1]], lens_k[[5, n - 1]] = most, 60
    cu_q, cu_k = starts(lens_q), starts(lens_k)
    q = rand((int(cu_q[-1]), H, D), 1).to(BF).cuda()
    kc, ks, kv = encode(rand((int(cu_k[-1]), H, D), 2), fp4)
    vc, vs, vv = encode(rand((int(cu_k[-1]), H, D), 3), fp4)
    o, lse = fwd(fp4)(q, kc, ks, vc, vs, causal=True, cu_q=torch.from_numpy(cu_q).cuda(),
                      cu_k=torch.from_numpy(cu_k).cuda(), max_q=most, max_k=60)
    some = np.flatnonzero(lens_q)
    compare(q, kv, vv, cu_q[some], cu_k[some], lens_q[some], lens_k[some], True, 1, D ** -0.5, o, lse)
