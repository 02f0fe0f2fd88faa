"""Softmax attention on the GPU (gdn_attn_fwd, gdn_attn_bwd) against the fp64
oracle's formulas (oracle/ops.py) on the same inputs.

Tolerances.  u = 2^-24, t the output type's half step (2^-8 for bf16, u for
fp32), b the half step of what is rounded between the products (2^-8 for bf16,
0 for fp32).  Per row, a score is off by at most
    E = max over its keys of  (D + 2) u scale sum|q k| + 4 u (|s| + max|s|) + 4 u,
so p = exp(s - lse) is off by 2 E relative (its own score, and the sum).  With n
terms added in fp32 (n u of the sum of sizes), and P and dS rounded by b:
    o:   (2 E + b + n u) sum p|v| + t |o|             lse: E + n u + 4 u |lse|
    dv:  sum_i p (2 E + b + n u) |do| + t |dv|
    dS:  e = p (2 E |dp - d| + (D + 2) u (sum|do v| + sum|do o|) + sum|do| e_o) + b |dS|
    dq:  scale sum_j (e + n u |dS|) |k| + t |dq|      dk: the same over i with |q|
where e_o is o's bound (the backward pass reads the rounded o).
"""
import numpy as np
import pytest
import torch

from gated_deltanet_scan_amd import api, autograd
from oracle import ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: U}


def host(t):
    return t.detach().double().cpu().numpy()


def dense(q, k, v, do, causal, block, scale, dtype):
    """(values, bars) of o, lse, dq, dk, dv for one sequence, from dense
    matrices (the oracle's row-by-row forms are checked against them below)."""
    lq, Hq, D = q.shape
    lk, Hk, _ = k.shape
    t, b = HALF[dtype], HALF[dtype] if dtype == BF else 0.0
    n = ops.visible(lq, lk, causal, block)
    see = np.arange(lk)[None, :] < n[:, None]
    val = dict(o=np.zeros_like(q), lse=np.full((lq, Hq), -np.inf), dq=np.zeros_like(q), dk=np.zeros_like(k),
               dv=np.zeros_like(v))
    bar = {x: np.zeros_like(y) for x, y in val.items()}
    if lq == 0:
        return val, bar
    for h in range(Hq):
        c = h * Hk // Hq
        qq, kk, vv, dd = q[:, h], k[:, c], v[:, c], do[:, h]
        s = np.where(see, scale * (qq @ kk.T), -np.inf)
        m = np.where(n > 0, s.max(-1, initial=-np.inf), 0.0)
        p = np.exp(s - m[:, None])
        l = p.sum(-1)
        p = p / np.where(l > 0, l, 1)[:, None]
        with np.errstate(divide="ignore"):
            lse = np.where(l > 0, m + np.log(l), -np.inf)
        sa = np.where(see, np.abs(s), 0.0)
        E = (np.where(see, (D + 2) * U * scale * (np.abs(qq) @ np.abs(kk).T) + 4 * U * sa, 0).max(-1, initial=0.0) +
             4 * U * sa.max(-1, initial=0.0) + 4 * U)
        o = p @ vv
        eo = (2 * E + b + lk * U)[:, None] * (p @ np.abs(vv)) + t * np.abs(o)
        val["o"][:, h], bar["o"][:, h] = o, eo
        val["lse"][:, h] = lse
        bar["lse"][:, h] = E + lk * U + 4 * U * np.where(np.isfinite(lse), np.abs(lse), 0)
        dp = dd @ vv.T
        delta = (dd * o).sum(-1, keepdims=True)
        ds = p * (dp - delta)
        e = p * (2 * E[:, None] * np.abs(dp - delta) +
                 (D + 2) * U * (np.abs(dd) @ np.abs(vv).T + (np.abs(dd) * np.abs(o)).sum(-1, keepdims=True)) +
                 (np.abs(dd) * eo).sum(-1, keepdims=True)) + b * np.abs(ds)
        val["dq"][:, h] = scale * (ds @ kk)
        bar["dq"][:, h] = scale * ((e + lk * U * np.abs(ds)) @ np.abs(kk)) + t * np.abs(val["dq"][:, h])
        val["dk"][:, c] += scale * (ds.T @ qq)
        bar["dk"][:, c] += scale * ((e + lq * Hq // Hk * U * np.abs(ds)).T @ np.abs(qq))
        val["dv"][:, c] += p.T @ dd
        bar["dv"][:, c] += (p * (2 * E + b + lq * Hq // Hk * U)[:, None]).T @ np.abs(dd)
    for x in ("dk", "dv"):
        bar[x] += t * np.abs(val[x])
    return val, bar


def starts(lens, gap=0):
    return np.concatenate([[0], np.cumsum([n + gap for n in lens])]).astype(np.int32)


def check(got, ref, bar, name):
    if got.size == 0:
        return
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine]), name
    err = np.abs(got[fine] - ref[fine])
    bar = bar[fine] + 1e-300
    print("%s: max err %.2e, most of the bar %.3f" % (name, err.max(initial=0), (err / bar).max(initial=0)))
    assert np.all(err <= bar), (name, (err / bar).max())


def inputs(cu_q, cu_k, Hq, Hk, D, dtype, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda n, h: (torch.randn((int(n), h, D), generator=g) * std).to(dtype).cuda()
    return mk(cu_q[-1], Hq), mk(cu_k[-1], Hk), mk(cu_k[-1], Hk), mk(cu_q[-1], Hq)


def compare(q, k, v, do, cu_q, cu_k, lens_q, lens_k, causal, block, scale, got, names):
    arrays = [host(x) for x in (q, k, v, do)]
    for s, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        a, c = slice(cu_q[s], cu_q[s] + lq), slice(cu_k[s], cu_k[s] + lk)
        val, bar = dense(arrays[0][a], arrays[1][c], arrays[2][c], arrays[3][a], causal, block, scale, q.dtype)
        for n, t in zip(names, got):
            z = c if n in ("dk", "dv") else a
            check(host(t[z.start:z.stop]), val[n], bar[n], "%s[%d]" % (n, s))


CASES = [
    # lens_q, lens_k, Hq, Hk, D, causal, block
    ([1], [1], 1, 1, 16, False, 1),
    ([1], [1], 4, 1, 128, True, 1),
    ([64], [64], 2, 2, 64, True, 1),
    ([65, 1, 0, 31], [65, 1, 5, 31], 4, 2, 32, True, 1),
    ([33, 7], [0, 300], 3, 3, 128, False, 1),
    ([100, 40], [37, 41], 2, 1, 64, True, 1),           # rows that see nothing
    ([130, 257], [130, 257], 2, 2, 128, True, 44),      # frames of 44 tokens, the last one short
    ([88], [300], 6, 2, 64, True, 88),                  # a new frame against a cache that ends inside a frame
    ([5], [1000], 8, 2, 128, True, 1),
    ([300], [300], 8, 1, 32, True, 7),
    ([200, 3, 129], [77, 700, 128], 4, 4, 128, False, 1),
    ([513], [513], 2, 1, 16, True, 1),
    ([700], [900], 4, 1, 128, True, 1),                 # many rows to a key head: rows split in the dk/dv kernel
    ([1100, 30], [1100, 30], 2, 1, 64, False, 1),
    ([290], [290], 3, 1, 64, True, 1),                  # heads that do not divide a row tile
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_packed_forward_and_backward(case, dtype):
    lens_q, lens_k, Hq, Hk, D, causal, block = CASES[case]
    cu_q, cu_k = starts(lens_q), starts(lens_k)
    q, k, v, do = inputs(cu_q, cu_k, Hq, Hk, D, dtype, seed=case)
    kw = dict(causal=causal, causal_block=block, cu_q=torch.from_numpy(cu_q).cuda(),
              cu_k=torch.from_numpy(cu_k).cuda(), max_q=max(lens_q), max_k=max(lens_k))
    o, lse = api.attention_fwd(q, k, v, **kw)
    grads = api.attention_bwd(q, k, v, o, lse, do, **kw)
    torch.cuda.synchronize()
    compare(q, k, v, do, cu_q, cu_k, lens_q, lens_k, causal, block, D ** -0.5, (o, lse, *grads),
            ("o", "lse", "dq", "dk", "dv"))


@pytest.mark.parametrize("n", [64, 65, 150])
def test_many_sequences(n):
    """More sequences than a wave has lanes, of several tiles or none."""
    r = np.random.default_rng(n)
    lens = [int(x) for x in r.choice([0, 1, 20, 64, 129, 300], n)]
    cu = starts(lens)
    q, k, v, do = inputs(cu, cu, 4, 2, 32, BF, seed=n)
    c = torch.from_numpy(cu).cuda()
    kw = dict(causal=True, cu_q=c, cu_k=c, max_q=300, max_k=300)
    o, lse = api.attention_fwd(q, k, v, **kw)
    grads = api.attention_bwd(q, k, v, o, lse, do, **kw)
    torch.cuda.synchronize()
    compare(q, k, v, do, cu, cu, lens, lens, True, 1, 32 ** -0.5, (o, lse, *grads), ("o", "lse", "dq", "dk", "dv"))


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with a workspace of its own."""
    sets = [inputs([0, 600], [0, 600], 4, 1, 128, BF, seed=s) for s in (20, 21)]
    ref = []
    for q, k, v, do in sets:
        o, lse = api.attention_fwd(q[None], k[None], v[None], causal=True)
        ref.append((o, lse, *api.attention_bwd(q[None], k[None], v[None], o, lse, do[None], causal=True)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(3):
        for i, ((q, k, v, do), s) in enumerate(zip(sets, streams)):
            o, lse = api.attention_fwd(q[None], k[None], v[None], causal=True, stream=s)
            got[i] = (o, lse, *api.attention_bwd(q[None], k[None], v[None], o, lse, do[None], causal=True, stream=s))
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_dense_form_is_the_oracle():
    r = np.random.default_rng(0)
    q, do = r.standard_normal((2, 9, 4, 8))
    k, v = r.standard_normal((2, 11, 2, 8))
    val, _ = dense(q, k, v, do, True, 3, 0.4, F32)
    o, lse = ops.attention(q, k, v, True, 3, 0.4)
    for a, b in zip((o, lse, *ops.attention_bwd(q, k, v, do, True, 3, 0.4)), val.values()):
        np.testing.assert_allclose(a, b, atol=1e-12)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lq,G,D", [(1, 4, 128), (1, 1, 64), (3, 8, 32), (17, 2, 128), (880, 1, 128)])
def test_cache_filled_in_part(lq, G, D, dtype):
    """Few queries against long caches with room: the keys are split over
    workgroups.  What lies behind a cache's length is NaN and must not matter."""
    lens_k = [lq, 2500, 0, 4096, 1025]
    room, Hk = 4100, 2
    cu_q = starts([lq] * 5)
    cu_k = (np.arange(6) * room).astype(np.int32)
    q, k, v, _ = inputs(cu_q, cu_k, Hk * G, Hk, D, dtype, seed=lq)
    for s, n in enumerate(lens_k):
        k[s * room + n:(s + 1) * room] = float("nan")
        v[s * room + n:(s + 1) * room] = float("nan")
    kl = torch.tensor(lens_k, dtype=torch.int32, device="cuda")
    for causal in (True, False):
        o, lse = api.attention_fwd(q.reshape(5, lq, Hk * G, D), k.reshape(5, room, Hk, D), v.reshape(5, room, Hk, D),
                                   causal=causal, k_len=kl)
        torch.cuda.synchronize()
        assert lse.shape == (5, lq, Hk * G)
        compare(q, k, v, torch.zeros_like(q), cu_q, cu_k, [lq] * 5, lens_k, causal, 1, D ** -0.5,
                (o.reshape(q.shape), lse.reshape(-1, Hk * G)), ("o", "lse"))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 32, 128])
def test_every_number_of_splits(D, dtype):
    """A single query against caches that take 1 to 70 splits, all remainders of
    the join's four-way sums and both sides of its 64-lane batches among them."""
    unit = 512 if dtype == BF and D > 16 else 128
    counts = [1, 2, 3, 4, 5, 15, 16, 17, 18, 19, 21, 34, 47, 58, 61, 62, 63, 64, 65, 66, 70]
    lens_k = [c * unit - (7 * c) % unit for c in counts]
    n, room = len(counts), 70 * unit
    cu_q, cu_k = starts([1] * n), (np.arange(n + 1) * room).astype(np.int32)
    q, k, v, _ = inputs(cu_q, cu_k, 2, 1, D, dtype, seed=D)
    kl = torch.tensor(lens_k, dtype=torch.int32, device="cuda")
    o, lse = api.attention_fwd(q[:, None], k.reshape(n, room, 1, D), v.reshape(n, room, 1, D), causal=True, k_len=kl)
    torch.cuda.synchronize()
    compare(q, k, v, torch.zeros_like(q), cu_q, cu_k, [1] * n, lens_k, True, 1, D ** -0.5,
            (o.reshape(q.shape), lse.reshape(-1, 2)), ("o", "lse"))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_frames_are_frame_causal(dtype):
    """[B, F, N, H, D]: causal means whole frames by default; every frame of a
    clip equals one streamed call of that frame against the frames so far."""
    B, F, N, H, D = 2, 4, 50, 2, 64
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((B, F, N, H, D), generator=g).to(dtype).cuda() for _ in range(3))
    o, lse = api.attention_fwd(q, k, v, causal=True)
    torch.cuda.synchronize()
    for b in range(B):
        val, bar = dense(*[host(t[b]).reshape(F * N, H, D) for t in (q, k, v)], np.zeros((F * N, H, D)), True, N,
                         D ** -0.5, dtype)
        check(host(o[b]).reshape(F * N, H, D), val["o"], bar["o"], "o")
    for f in range(F):
        of, _ = api.attention_fwd(q[:, f].contiguous(), k.reshape(B, F * N, H, D)[:, :(f + 1) * N],
                                  v.reshape(B, F * N, H, D)[:, :(f + 1) * N], causal=True, causal_block=N)
        torch.cuda.synchronize()
        for b in range(B):
            val, bar = dense(host(q[b, f]), *[host(t[b, :f + 1]).reshape(-1, H, D) for t in (k, v)],
                             np.zeros((N, H, D)), True, N, D ** -0.5, dtype)
            check(host(of[b]), val["o"], bar["o"], "o of frame %d" % f)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_strided_views_and_scale(dtype):
    """q, k and v as slices of one fused projection, and a scale of the caller's."""
    B, L, Hq, Hk, D = 2, 70, 4, 2, 64
    fused = torch.randn((B, L, Hq + 2 * Hk, D), generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    q, k, v = fused[:, :, :Hq], fused[:, :, Hq:Hq + Hk], fused[:, :, Hq + Hk:]
    do = torch.randn((B, L, Hq, D), device="cuda").to(dtype)
    kw = dict(causal=True, scale=0.3)
    o, lse = api.attention_fwd(q, k, v, **kw)
    g = api.attention_bwd(q, k, v, o, lse, do, **kw)
    qc, kc, vc = (t.contiguous() for t in (q, k, v))
    o2, lse2 = api.attention_fwd(qc, kc, vc, **kw)
    g2 = api.attention_bwd(qc, kc, vc, o2, lse2, do, **kw)
    torch.cuda.synchronize()
    for x, y in zip((o, lse, *g), (o2, lse2, *g2)):
        assert torch.equal(x, y)
    for b in range(B):
        val, bar = dense(*[host(t[b]) for t in (q, k, v, do)], True, 1, 0.3, dtype)
        for n, t in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *g)):
            check(host(t[b]), val[n], bar[n], n)
    # the first tokens of a cache's slots: gradients come packed
    room = torch.full((B, L + 30, Hk, D), float("nan"), device="cuda").to(dtype)
    kr, vr = room.clone(), room.clone()
    kr[:, :L], vr[:, :L] = kc, vc
    o3, lse3 = api.attention_fwd(qc, kr[:, :L], vr[:, :L], **kw)
    g3 = api.attention_bwd(qc, kr[:, :L], vr[:, :L], o3, lse3, do, **kw)
    torch.cuda.synchronize()
    for x, y in zip((o3, lse3, *g3), (o2, lse2, *g2)):
        assert torch.equal(x, y)
    with pytest.raises(ValueError, match="packed heads"):
        api.attention_fwd(qc.transpose(1, 2).contiguous().transpose(1, 2), kc, vc)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_large_scores(dtype):
    """Scores of several hundred: the running maximum moves, most weights vanish."""
    q, k, v, do = inputs([0, 150], [0, 150], 2, 2, 64, dtype, seed=5, std=6.0)
    args = [t.unsqueeze(0) for t in (q, k, v)]
    o, lse = api.attention_fwd(*args, causal=True)
    torch.cuda.synchronize()
    compare(q, k, v, do, [0], [0], [150], [150], True, 1, 0.125, (o[0], lse[0]), ("o", "lse"))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_tokens_of_no_sequence_are_left_alone(dtype):
    """Rows before, between and behind the sequences keep what they held."""
    q, k, v, do = inputs([0, 200], [0, 200], 2, 2, 64, dtype, seed=6)
    q[150:], k[150:], v[150:], do[150:] = [float("nan")] * 4
    cu = torch.tensor([10, 60, 60, 150], dtype=torch.int32, device="cuda")
    kw = dict(causal=True, cu_q=cu, max_q=90, max_k=90)
    o, lse = torch.full_like(q, 7), torch.full((200, 2), 7.0, device="cuda")
    grads = [torch.full_like(t, 7) for t in (q, k, v)]
    api.attention_fwd(q, k, v, o=o, lse=lse, **kw)
    api.attention_bwd(q, k, v, o, lse, do, dq=grads[0], dk=grads[1], dv=grads[2], **kw)
    torch.cuda.synchronize()
    for t in (o, lse, *grads):
        assert (t[:10] == 7).all() and (t[150:] == 7).all()
    compare(q, k, v, do, [10, 60], [10, 60], [50, 90], [50, 90], True, 1, 0.125, (o, lse, *grads),
            ("o", "lse", "dq", "dk", "dv"))


def test_offsets_out_of_range_are_clamped():
    """Offsets that point outside the tensors, run backwards or exceed max_q
    are cut on the device; what remains in range is computed."""
    q, k, v, do = inputs([0, 100], [0, 100], 2, 1, 64, BF, seed=7)
    cu = torch.tensor([-50, 40, 30, 1 << 30], dtype=torch.int32, device="cuda")
    kw = dict(cu_q=cu, max_q=64, max_k=64)
    o, lse = api.attention_fwd(q, k, v, **kw)
    api.attention_bwd(q, k, v, o, lse, do, **kw)
    torch.cuda.synchronize()
    # [0, 40), then nothing, then [30, 94): the first 30 rows belong to the first alone
    val, bar = dense(*[host(t[:40]) for t in (q, k, v, do)], False, 1, 0.125, BF)
    check(host(o[:30]), val["o"][:30], bar["o"][:30], "o")
    val, bar = dense(*[host(t[30:94]) for t in (q, k, v, do)], False, 1, 0.125, BF)
    check(host(o[40:94]), val["o"][10:], bar["o"][10:], "o")


def test_same_bits_every_time_and_in_graphs():
    """Two captured graphs that share one workspace, replayed in turn."""
    lens = [700, 1, 333]
    cu_h = starts(lens)
    cu = torch.from_numpy(cu_h).cuda()
    sets = [inputs(cu_h, cu_h, 4, 2, 128, BF, seed=s) for s in (8, 9)]
    kw = dict(causal=True, cu_q=cu, max_q=700, max_k=700)
    token = dict(causal=True)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    ref, outs, graphs = [], [], []
    for q, k, v, do in sets:
        o, lse = api.attention_fwd(q, k, v, **kw)
        t, tl = api.attention_fwd(q[None, :1], k[None], v[None], **token)
        ref.append((o, lse, *api.attention_bwd(q, k, v, o, lse, do, **kw), t, tl))
    torch.cuda.synchronize()
    for (q, k, v, do), r in zip(sets, ref):
        out = [torch.empty_like(x) for x in r]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.attention_fwd(q, k, v, o=out[0], lse=out[1], workspace=ws, **kw)
            api.attention_bwd(q, k, v, out[0], out[1], do, dq=out[2], dk=out[3], dv=out[4], workspace=ws, **kw)
            api.attention_fwd(q[None, :1], k[None], v[None], o=out[5], lse=out[6], workspace=ws, **token)
        outs.append(out)
        graphs.append(g)
    for _ in range(3):
        for out in outs:
            for x in out:
                x.zero_()
        ws.fill_(255)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out, r in zip(outs, ref):
            for x, y in zip(out, r):
                assert torch.equal(x, y)


def test_side_stream():
    q, k, v, _ = inputs([0, 300], [0, 300], 2, 2, 128, BF, seed=10)
    ref = api.attention_fwd(q[None], k[None], v[None])[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = api.attention_fwd(q[None], k[None], v[None], stream=s)[0]
    s.synchronize()
    assert torch.equal(o, ref)


def test_empty():
    q, k, v, do = inputs([0, 5], [0, 5], 2, 2, 64, BF)
    o, lse = api.attention_fwd(q[None, :0], k[None], v[None])
    assert o.shape == (1, 0, 2, 64) and lse.shape == (1, 0, 2)
    dq, dk, dv = api.attention_bwd(q[None, :0], k[None], v[None], o, lse, do[None, :0])
    torch.cuda.synchronize()
    assert not dk.any() and not dv.any()
    o, lse = api.attention_fwd(q[None], k[None, :0], v[None, :0])
    torch.cuda.synchronize()
    assert not o.any() and torch.isneginf(lse).all()


def test_autograd():
    lens = [40, 90]
    cu_h = starts(lens)
    cu = torch.from_numpy(cu_h).cuda()
    q, k, v, do = inputs([0, 140], [0, 140], 4, 2, 64, BF, seed=11)          # ten tokens of no sequence
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    kw = dict(causal=True, max_q=90, max_k=90)
    o = autograd.attention(*leaves, cu_q=cu, **kw)
    o.backward(do)
    o0, lse = api.attention_fwd(q, k, v, cu_q=cu, **kw)
    ref = api.attention_bwd(q, k, v, o0, lse, do, cu_q=cu, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o[:130], o0[:130]) and not o[130:].any()
    for a, r in zip(leaves, ref):
        assert torch.equal(a.grad[:130], r[:130]) and not a.grad[130:].any()


def test_gradient_against_differences():
    """Directional differences of the oracle's forward at the kernel's fp32
    inputs: a step of 1e-4 leaves about 1e-8 relative, the kernel 1e-6."""
    q, k, v, do = inputs([0, 20], [0, 24], 4, 2, 32, F32, seed=12)
    o, lse = api.attention_fwd(q[None], k[None], v[None], causal=True)
    grads = [host(t[0]) for t in api.attention_bwd(q[None], k[None], v[None], o, lse, do[None], causal=True)]
    args = [host(t) for t in (q, k, v)]
    r = np.random.default_rng(0)
    for i, g in enumerate(grads):
        d = r.standard_normal(args[i].shape)
        val = []
        for h in (1e-4, -1e-4):
            a = list(args)
            a[i] = a[i] + h * d
            val.append((ops.attention(*a, causal=True)[0] * host(do)).sum())
        assert abs((val[0] - val[1]) / 2e-4 - (g * d).sum()) <= 1e-5 * np.linalg.norm(g) * np.linalg.norm(d)


def test_long_cache_offsets_past_32_bits():
    """A cache whose last keys lie more than 2^32 bytes into the tensor."""
    Hk, D, room = 8, 128, 1100000                       # 2.25 GB a sequence
    k = torch.zeros((2, room, Hk, D), dtype=BF, device="cuda")
    v = torch.zeros((2, room, Hk, D), dtype=BF, device="cuda")
    n = 300
    g = torch.Generator().manual_seed(13)
    kk, vv, q = (torch.randn((n, h, D), generator=g).to(BF).cuda() for h in (Hk, Hk, Hk))
    k[1, room - n:], v[1, room - n:] = kk, vv
    kf, vf = k.reshape(-1, Hk, D), v.reshape(-1, Hk, D)
    cu_q = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([2 * room - n, 2 * room], dtype=torch.int32, device="cuda")
    o, lse = api.attention_fwd(q[:1], kf, vf, cu_q=cu_q, cu_k=cu_k, max_q=1, max_k=n, causal=True)
    torch.cuda.synchronize()
    compare(q[:1], kk, vv, q[:1], [0], [0], [1], [n], True, 1, D ** -0.5, (o, lse), ("o", "lse"))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_thousands_of_sequences(dtype):
    """More sequences than one step of the tile search takes, a few of them of
    several tiles."""
    n = 1300
    lens = [(3, 0, 1, 2)[i % 4] for i in range(n)]
    for i in (0, 511, 512, 777, n - 1):
        lens[i] = 150
    cu = starts(lens)
    q, k, v, do = inputs(cu, cu, 2, 1, 32, dtype, seed=n)
    kw = dict(causal=True, cu_q=torch.from_numpy(cu).cuda(), max_q=150, max_k=150)
    o, lse = api.attention_fwd(q, k, v, **kw)
    grads = api.attention_bwd(q, k, v, o, lse, do, **kw)
    torch.cuda.synchronize()
    compare(q, k, v, do, cu, cu, lens, lens, True, 1, 32 ** -0.5, (o, lse, *grads), ("o", "lse", "dq", "dk", "dv"))


def test_bounds_past_the_tensors():
    """max_q, max_k and causal_block of more than 32 bits mean all tokens."""
    q, k, v, do = inputs([0, 200], [0, 200], 2, 2, 32, BF, seed=3)
    cu = torch.tensor([0, 80, 200], dtype=torch.int32, device="cuda")
    a = api.attention_fwd(q, k, v, cu_q=cu, causal=True, causal_block=2 ** 32 + 1, max_q=2 ** 32 + 1, max_k=2 ** 40)
    b = api.attention_fwd(q, k, v, cu_q=cu, max_q=120, max_k=120)
    torch.cuda.synchronize()
    compare(q, k, v, do, [0, 80], [0, 80], [80, 120], [80, 120], False, 1, 32 ** -0.5, a, ("o", "lse"))
    compare(q, k, v, do, [0, 80], [0, 80], [80, 120], [80, 120], False, 1, 32 ** -0.5, b, ("o", "lse"))
