"""Infinities and NaN in softmax attention (gdn_attn_fwd, gdn_attn_bwd): a row
that must not see such a value gives what it gives without it, within the bars
of tests/test_gpu_attention.py, forward and backward; a row that sees it is not
finite where the formula says so."""
import numpy as np
import pytest
import torch

from gated_deltanet_scan_amd import api
from oracle import ops
from test_gpu_attention import BF, F32, dense, host, inputs

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
SHAPES = [
    # lq, lk, Hq, Hk, block, D
    (200, 200, 4, 2, 1, 128),
    (150, 300, 2, 2, 44, 64),
    (70, 40, 8, 2, 1, 32),           # rows that see nothing
    (300, 300, 2, 2, 7, 16),
    (5, 2000, 4, 2, 1, 128),         # split keys
    (700, 900, 8, 2, 1, 64),         # split rows in the dk/dv kernel
    (300, 300, 4, 2, 100, 128),      # 256 rows to a workgroup
]


def near(got, val, bar, keep, name):
    """`got` within the bars on the rows [n, H] of `keep`."""
    g, v, b = got[keep], val[keep], bar[keep]
    fine = np.isfinite(v)
    assert np.array_equal(g[~fine], v[~fine]), name
    assert np.isfinite(g[fine]).all(), name
    assert (np.abs(g[fine] - v[fine]) <= b[fine] + 1e-300).all(), name


def run(q, k, v, do, kw):
    o, lse = api.attention_fwd(*(t[None] for t in (q, k, v)), **kw)
    dq, dk, dv = api.attention_bwd(*(t[None] for t in (q, k, v)), o, lse, do[None], **kw)
    torch.cuda.synchronize()
    return {n: host(t[0]) for n, t in dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv).items()}


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_stays_with_the_rows_that_see_it(shape, dtype):
    lq, lk, Hq, Hk, block, D = shape
    G = Hq // Hk
    q, k, v, do = inputs([0, lq], [0, lk], Hq, Hk, D, dtype, seed=lq)
    kw = dict(causal=True, causal_block=block)
    n = ops.visible(lq, lk, True, block)
    val, bar = dense(*[host(t) for t in (q, k, v, do)], True, block, D ** -0.5, dtype)
    mine = np.arange(Hq)[None, :] < G                         # heads that share key head 0
    key0 = np.arange(Hk)[None, :] == 0
    # two keys near the end, hidden from the rows before them
    ja, jb = lk - 2, lk - min(4, lk)
    sees = (n[:, None] > min(ja, jb)) & mine                  # [lq, Hq]

    # values: one feature each
    vx = v.clone()
    vx[ja, 0, 3], vx[jb, 0, 5] = NAN, INF
    got = run(q, k, vx, do, kw)
    near(got["lse"], val["lse"], bar["lse"], np.ones_like(sees), "lse")
    near(got["o"], val["o"], bar["o"], ~sees, "o")
    rest = [d for d in range(D) if d not in (3, 5)]
    near(got["o"][..., rest], val["o"][..., rest], bar["o"][..., rest], sees, "o")
    assert not np.isfinite(got["o"][..., 3][(n[:, None] > ja) & mine]).any()
    assert not np.isfinite(got["o"][..., 5][(n[:, None] > jb) & mine]).any()
    near(got["dq"], val["dq"], bar["dq"], ~sees, "dq")
    assert not np.isfinite(got["dq"][sees]).any()
    near(got["dk"], val["dk"], bar["dk"], np.broadcast_to(~key0, (lk, Hk)), "dk")
    near(got["dv"], val["dv"], bar["dv"], np.ones((lk, Hk), bool), "dv")

    # a key
    kx = k.clone()
    kx[ja, 0, 1] = NAN
    sees = (n[:, None] > ja) & mine
    got = run(q, kx, v, do, kw)
    for x in ("o", "lse", "dq"):
        near(got[x], val[x], bar[x], ~sees, x)
        assert not np.isfinite(got[x][sees]).any()
    for x in ("dk", "dv"):
        near(got[x], val[x], bar[x], np.broadcast_to(~key0, (lk, Hk)), x)

    # a query and its gradient, the first row that sees something of a block
    i0 = int(np.argmax(n > 0))
    qx, dx = q.clone(), do.clone()
    qx[i0, 0], dx[i0, 0, 2] = NAN, INF
    qx[:i0], dx[:i0] = NAN, NAN                               # rows that see nothing take no part
    row = (np.arange(lq)[:, None] == i0) & (np.arange(Hq)[None, :] == 0)
    hit = (np.arange(lk)[:, None] < n[i0]) & key0
    got = run(qx, k, v, dx, kw)
    for x in ("o", "lse", "dq"):
        near(got[x], val[x], bar[x], ~row, x)
        assert not np.isfinite(got[x][row]).any()
    for x in ("dk", "dv"):
        near(got[x], val[x], bar[x], ~hit, x)
        assert not np.isfinite(got[x][hit]).any()
