"""Softmax attention over MXFP8 and MXFP4 caches (gdn_attn_fwd_fp8, gdn_attn_fwd_fp4)
against the fp64 oracle's formulas on the dequantised values, within the bars of
tests/test_gpu_attention.py for bf16 (codes widen to bf16 exactly, so nothing else is
rounded)."""
import numpy as np
import pytest
import torch

from gated_deltanet_scan_amd import api, inputs
from oracle import ops
from test_gpu_attention import BF, check, dense, host, starts

pytestmark = pytest.mark.gpu

NAN = float("nan")
FORMATS = pytest.mark.parametrize("fp4", [True, False], ids=["fp4", "fp8"])


def rand(shape, seed, std=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std


def encode(x, fp4):
    """(codes, scales, values) on the device; the values in float64 on the host."""
    c, s, v = (inputs.to_mxfp4 if fp4 else inputs.to_mxfp8)(x.numpy())
    c = torch.from_numpy(c).cuda()
    return (c if fp4 else c.view(torch.float8_e4m3fn)), torch.from_numpy(s).cuda(), v.astype(np.float64)


def fwd(fp4):
    return api.attention_fwd_fp4 if fp4 else api.attention_fwd_fp8


def compare(q, kv, vv, cu_q, cu_k, lens_q, lens_k, causal, block, scale, o, lse):
    for s, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        a, c = slice(cu_q[s], cu_q[s] + lq), slice(cu_k[s], cu_k[s] + lk)
        x = host(q[a.start:a.stop])
        val, bar = dense(x, kv[c], vv[c], np.zeros_like(x), causal, block, scale, BF)
        check(host(o[a.start:a.stop]), val["o"], bar["o"], "o[%d]" % s)
        check(host(lse[a.start:a.stop]), val["lse"], bar["lse"], "lse[%d]" % s)


CASES = [
    # lens_q, lens_k, Hq, Hk, D, causal, block
    ([1], [1], 1, 1, 32, False, 1),
    ([1], [1], 4, 1, 128, True, 1),
    ([64], [64], 2, 2, 64, True, 1),
    ([65, 1, 0, 31], [65, 1, 5, 31], 4, 2, 32, True, 1),
    ([33, 7], [0, 300], 3, 3, 128, False, 1),
    ([100, 40], [37, 41], 2, 1, 64, True, 1),           # rows that see nothing
    ([130, 257], [130, 257], 2, 2, 128, True, 44),      # frames of 44 tokens, the last one short
    ([88], [300], 6, 2, 64, True, 88),
    ([5], [1000], 8, 2, 128, True, 1),
    ([200, 3, 129], [77, 700, 128], 4, 4, 128, False, 1),
    ([290], [290], 3, 1, 64, True, 1),                  # heads that do not divide a row tile
    ([300], [300], 4, 2, 128, True, 100),               # 256 rows to a workgroup
    ([1, 1, 1], [700, 33, 64], 32, 8, 128, True, 1),
    ([2, 3, 1], [2500, 5, 1], 8, 8, 64, True, 1),
    ([4], [31], 4, 1, 32, False, 1),
    ([1, 1], [65, 129], 16, 1, 128, True, 1),           # sixteen heads on one
    ([1, 2], [700, 90], 24, 2, 64, True, 1),            # twelve
    ([1, 1], [400, 17], 7, 7, 128, True, 1),
    ([1, 1], [400, 17], 5, 5, 32, True, 1),
    ([17, 1], [400, 17], 3, 3, 64, True, 1),
]


@FORMATS
@pytest.mark.parametrize("case", range(len(CASES)))
def test_packed(case, fp4):
    lens_q, lens_k, Hq, Hk, D, causal, block = CASES[case]
    cu_q, cu_k = starts(lens_q), starts(lens_k)
    q = rand((int(cu_q[-1]), Hq, D), case).to(BF).cuda()
    kc, ks, kv = encode(rand((int(cu_k[-1]), Hk, D), case + 100), fp4)
    vc, vs, vv = encode(rand((int(cu_k[-1]), Hk, D), case + 200), fp4)
    o, lse = fwd(fp4)(q, kc, ks, vc, vs, causal=causal, causal_block=block, cu_q=torch.from_numpy(cu_q).cuda(),
                      cu_k=torch.from_numpy(cu_k).cuda(), max_q=max(lens_q), max_k=max(lens_k))
    torch.cuda.synchronize()
    compare(q, kv, vv, cu_q, cu_k, lens_q, lens_k, causal, block, D ** -0.5, o, lse)


@FORMATS
@pytest.mark.parametrize("n", [64, 65, 150])
def test_many_sequences(n, fp4):
    r = np.random.default_rng(n)
    lens_q = [int(x) for x in r.choice([0, 1, 1, 3, 40], n)]
    lens_k = [int(x) for x in r.choice([0, 1, 20, 64, 129, 300], n)]
    cu_q, cu_k = starts(lens_q), starts(lens_k)
    q = rand((int(cu_q[-1]), 4, 32), n).to(BF).cuda()
    kc, ks, kv = encode(rand((int(cu_k[-1]), 2, 32), n + 1), fp4)
    vc, vs, vv = encode(rand((int(cu_k[-1]), 2, 32), n + 2), fp4)
    o, lse = fwd(fp4)(q, kc, ks, vc, vs, causal=True, cu_q=torch.from_numpy(cu_q).cuda(),
                      cu_k=torch.from_numpy(cu_k).cuda(), max_q=40, max_k=300)
    torch.cuda.synchronize()
    compare(q, kv, vv, cu_q, cu_k, lens_q, lens_k, True, 1, 32 ** -0.5, o, lse)


@FORMATS
@pytest.mark.parametrize("lq,G,Hk,D", [(1, 4, 2, 128), (1, 1, 3, 64), (3, 8, 2, 32), (17, 2, 2, 128), (880, 1, 2, 128),
                                       (1, 4, 8, 128), (4, 4, 1, 64), (1, 32, 1, 128), (1, 1, 16, 64)])
def test_cache_filled_in_part(lq, G, Hk, D, fp4):
    """Few queries against long caches with room (the keys are split over workgroups).  What lies behind a cache's
    length is NaN and must not matter."""
    lens_k = [lq, 2500, 0, 4096, 1025]
    room = 4100
    q = rand((5, lq, G * Hk, D), 1).to(BF).cuda()
    kc, ks, kv = encode(rand((5, room, Hk, D), 2), fp4)
    vc, vs, vv = encode(rand((5, room, Hk, D), 3), fp4)
    for b, n in enumerate(lens_k):
        ks[b, n:] = 255
        vs[b, n:] = 255
        kc.view(torch.uint8)[b, n:] = 255
    n = torch.tensor(lens_k, dtype=torch.int32, device="cuda")
    o, lse = fwd(fp4)(q, kc, ks, vc, vs, causal=True, k_len=n)
    part = [t[:, :4096] for t in (kc, ks, vc, vs)]                # the same slots, cut
    o2, lse2 = fwd(fp4)(q, *part, causal=True, k_len=n)
    torch.cuda.synchronize()
    for b, lk in enumerate(lens_k):
        x = host(q[b])
        val, bar = dense(x, kv[b, :lk], vv[b, :lk], np.zeros_like(x), True, 1, D ** -0.5, BF)
        for oo, ll in ((o, lse), (o2, lse2)):
            check(host(oo[b]), val["o"], bar["o"], "o[%d]" % b)
            check(host(ll[b]), val["lse"], bar["lse"], "lse[%d]" % b)


@FORMATS
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("lq,block,G,Hk,D", [(6, 3, 2, 3, 64), (7, 4, 4, 2, 128), (16, 16, 2, 1, 32), (9, 2, 1, 8, 128),
                                             (60, 7, 2, 2, 64)])
def test_blocks_over_a_part_of_the_cache(lq, block, G, Hk, D, causal, fp4):
    """Drafts of several blocks, and full attention, over caches whose places behind their length are NaN: lengths
    that end inside a step, at its end, short of the queries, and of several splits."""
    lens_k = [lq, 64, 0, 1500, 3, 2049, 96]
    room, B = 2100, 7
    q = rand((B, lq, G * Hk, D), 1).to(BF).cuda()
    kc, ks, kv = encode(rand((B, room, Hk, D), 2), fp4)
    vc, vs, vv = encode(rand((B, room, Hk, D), 3), fp4)
    for b, n in enumerate(lens_k):
        ks[b, n:] = 255
        vs[b, n:] = 255
        vc.view(torch.uint8)[b, n:] = 255
    n = torch.tensor(lens_k, dtype=torch.int32, device="cuda")
    o, lse = fwd(fp4)(q, kc, ks, vc, vs, causal=causal, causal_block=block, k_len=n)
    for b, lk in enumerate(lens_k):
        x = host(q[b])
        val, bar = dense(x, kv[b, :lk], vv[b, :lk], np.zeros_like(x), causal, block, D ** -0.5, BF)
        check(host(o[b]), val["o"], bar["o"], "o[%d]" % b)
        check(host(lse[b]), val["lse"], bar["lse"], "lse[%d]" % b)


@FORMATS
@pytest.mark.parametrize("lk,Hq,Hk,D", [(40001, 4, 1, 32), (33000, 16, 1, 128), (17000, 2, 2, 64)])
def test_many_splits(lk, Hq, Hk, D, fp4):
    """One request against a long cache: hundreds of splits to a row."""
    q = rand((1, 1, Hq, D), 1).to(BF).cuda()
    kc, ks, kv = encode(rand((1, lk, Hk, D), 2), fp4)
    vc, vs, vv = encode(rand((1, lk, Hk, D), 3), fp4)
    for causal in (True, False):
        o, lse = fwd(fp4)(q, kc, ks, vc, vs, causal=causal)
        x = host(q[0])
        val, bar = dense(x, kv[0], vv[0], np.zeros_like(x), causal, 1, D ** -0.5, BF)
        check(host(o[0]), val["o"], bar["o"], "o")
        check(host(lse[0]), val["lse"], bar["lse"], "lse")


@FORMATS
@pytest.mark.parametrize("lq,lk,Hq,Hk,block,D", [(200, 200, 4, 2, 1, 128), (150, 300, 2, 2, 44, 64), (70, 40, 8, 2, 1, 32),
                                                 (5, 2000, 4, 2, 1, 128), (300, 300, 4, 2, 100, 128),
                                                 (3, 900, 4, 2, 1, 64), (8, 8, 4, 2, 1, 32)])
def test_nan_stays_with_the_rows_that_see_it(lq, lk, Hq, Hk, block, D, fp4):
    q = rand((lq, Hq, D), lq).to(BF).cuda()
    kc, ks, kv = encode(rand((lk, Hk, D), lq + 1), fp4)
    vc, vs, vv = encode(rand((lk, Hk, D), lq + 2), fp4)
    n = ops.visible(lq, lk, True, block)
    G = Hq // Hk
    mine = np.arange(Hq)[None, :] < G                            # heads that share key head 0
    val, bar = dense(host(q), kv, vv, np.zeros((lq, Hq, D)), True, block, D ** -0.5, BF)
    ja, jb = lk - 2, lk - min(4, lk)
    for which in ("k", "v"):
        k2, v2 = ks.clone(), vs.clone()
        for j in (ja, jb):
            (k2 if which == "k" else v2)[j, 0, 0] = 255
        o, lse = fwd(fp4)(q[None], kc[None], k2[None], vc[None], v2[None], causal=True, causal_block=block)
        o, lse = host(o[0]), host(lse[0])
        sees = (n[:, None] > min(ja, jb)) & mine
        fine = ~sees if which == "k" else ~sees[:, :, None] | (np.arange(D) >= 32)[None, None, :]
        ok = np.broadcast_to(fine[..., None] if which == "k" else fine, o.shape)
        assert np.isfinite(o[ok]).all() and np.all(np.abs(o - val["o"])[ok] <= bar["o"][ok] + 1e-300)
        assert np.isnan(o[~ok]).all()
        keep = ~sees if which == "k" else np.ones_like(sees)
        got, want = lse[keep], val["lse"][keep]
        some = np.isfinite(want)
        assert np.array_equal(got[~some], want[~some])
        assert np.all(np.abs(got[some] - want[some]) <= bar["lse"][keep][some])


@FORMATS
def test_scales_and_large_scores(fp4):
    """Scores of hundreds, blocks of very different scales, and a scale argument."""
    q = rand((1, 40, 4, 64), 1, 8.0).to(BF).cuda()
    k = rand((1, 300, 2, 64), 2, 1.0) * torch.exp2(torch.randint(-6, 4, (1, 300, 2, 2), generator=torch.Generator().manual_seed(5)).float()).repeat_interleave(32, -1)
    kc, ks, kv = encode(k, fp4)
    vc, vs, vv = encode(rand((1, 300, 2, 64), 3, 100.0), fp4)
    for scale in (0.125, 1.0, 1e-3):
        o, lse = fwd(fp4)(q, kc, ks, vc, vs, causal=True, scale=scale)
        x = host(q[0])
        val, bar = dense(x, kv[0], vv[0], np.zeros_like(x), True, 1, scale, BF)
        # a probability below fp32's least normal number is 0: off by less than 2^-126, times |v|, for each key
        check(host(o[0]), val["o"], bar["o"] + 300 * 2.0 ** -126 * np.abs(vv).max(), "o")
        check(host(lse[0]), val["lse"], bar["lse"], "lse")


@FORMATS
def test_near_the_bf16_kernels(fp4):
    """Frames [B, F, N, H, D] on the default mask, a query slice of a fused projection, against attention_fwd on the
    dequantised values: both round the same products, so they differ by a few of o's steps."""
    B, F, N, H, D = 2, 3, 50, 4, 128
    fused = rand((B, F, N, 3, H, D), 1).to(BF).cuda()
    kc, ks, kv = encode(rand((B, 4 * N, H, D), 2), fp4)
    vc, vs, vv = encode(rand((B, 4 * N, H, D), 3), fp4)
    q = fused[:, :, :, 1]
    o, lse = fwd(fp4)(q, kc, ks, vc, vs, causal=True)
    k, v = api.cache_read(kc, ks, vc, vs)
    ref, rl = api.attention_fwd(q.reshape(B, F * N, H, D).contiguous(), k, v, causal=True, causal_block=N)
    d = (o.reshape(ref.shape).double() - ref.double()).norm() / ref.double().norm()
    assert d <= 2 * 2.5e-3                                       # each is 2.5e-3 from 64 bits
    assert torch.allclose(lse.reshape(rl.shape), rl, rtol=0, atol=1e-4)


@FORMATS
def test_rows_behind_the_last_sequence(fp4):
    """Tokens of no sequence keep what o and lse hold; given outputs, a side stream, no lse."""
    cu = torch.tensor([2, 5, 5, 9], dtype=torch.int32, device="cuda")
    q = rand((12, 4, 64), 1).to(BF).cuda()
    kc, ks, _ = encode(rand((12, 2, 64), 2), fp4)
    vc, vs, _ = encode(rand((12, 2, 64), 3), fp4)
    kw = dict(causal=True, cu_q=cu, max_q=4, max_k=4)
    ref, rl = fwd(fp4)(q, kc, ks, vc, vs, **kw)
    o, lse = torch.full_like(q, 7.0), torch.full((12, 4), 7.0, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fwd(fp4)(q, kc, ks, vc, vs, o=o, lse=lse, stream=side, **kw)
    torch.cuda.synchronize()
    assert got[0] is o and got[1] is lse
    inside = torch.zeros(12, dtype=torch.bool)
    inside[2:9] = True
    assert torch.equal(o[inside], ref[inside]) and torch.equal(lse[inside], rl[inside])
    assert torch.all(o[~inside] == 7) and torch.all(lse[~inside] == 7)
    assert fwd(fp4)(q, kc, ks, vc, vs, return_lse=False, **kw)[1] is None


@FORMATS
@pytest.mark.parametrize("lq", [1, 100])
def test_two_streams_and_repeats(lq, fp4):
    """Calls that overlap on two streams give what they give alone, every time."""
    sets = []
    for s in (1, 2):
        q = rand((2, lq, 8, 128), s).to(BF).cuda()
        kc, ks, _ = encode(rand((2, 3000, 2, 128), s + 10), fp4)
        vc, vs, _ = encode(rand((2, 3000, 2, 128), s + 20), fp4)
        sets.append((q, kc, ks, vc, vs))
    ref = [fwd(fp4)(*x, causal=True) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [fwd(fp4)(*x, causal=True, stream=s) for x, s in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@FORMATS
@pytest.mark.parametrize("lq,block", [(4, 1), (4, 4), (40, 1)])
def test_lengths_past_the_slot(lq, block, fp4):
    """Tokens written and queried with the same lengths.  Within the slot a query lies where its token does; a length
    past it is the slot's size to attention, while tokens that find no room are dropped."""
    B, L, H, D = 4, 70, 2, 64
    n = [lq, L - 1, L, L + 3]
    old, new = rand((B, L, H, D), 1).to(BF), rand((B, lq, H, D), 2).to(BF)
    q = rand((B, lq, 2 * H, D), 3).to(BF).cuda()
    cache = api.cache_empty(B, L, H=H, D=D, fp4=fp4)
    api.cache_write(old.cuda(), old.cuda(), *cache)
    k_len = torch.tensor(n, dtype=torch.int32, device="cuda")
    api.cache_write(new.cuda(), new.cuda(), *cache, k_len=k_len)
    o, lse = fwd(fp4)(q, *cache, causal=True, causal_block=block, k_len=k_len)
    for b, m in enumerate(n):
        held = old[b].clone()
        room = min(lq, L - (m - lq))
        held[m - lq:m - lq + room] = new[b, :room]
        x, lk = encode(held.float(), fp4)[2], min(m, L)
        val, bar = dense(host(q[b]), x[:lk], x[:lk], np.zeros((lq, 2 * H, D)), True, block, D ** -0.5, BF)
        check(host(o[b]), val["o"], bar["o"], "o[%d]" % b)
        check(host(lse[b]), val["lse"], bar["lse"], "lse[%d]" % b)
