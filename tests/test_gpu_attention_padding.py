"""The places of a tile past a sequence's last row or key, in the backward pass:
whatever their scores come to, they change neither the gradients nor the way in
which they are computed.
"""
import pytest
import torch

from gated_deltanet_scan_amd import api

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("L", [40, 100])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_keys_past_the_end(D, L):
    """Scores of about -110: the logarithm of a row's sum is so low that a place
    without a key (score 0) would have a probability past fp32.  Tokens appended
    up to a whole tile, whose d_o is 0, add exact zeros to the gradients of the
    first L, so these have the same bits with and without them; sums formed
    again element by element (for places that are not finite) would not."""
    g = torch.Generator().manual_seed(D + L)
    whole, c = (L + 63) // 64 * 64, (110 / D ** 0.5) ** 0.5
    q, k, v, do = [torch.randn((1, whole, h, D), generator=g) for h in (4, 2, 2, 4)]
    q, k, do[:, L:] = c + 0.1 * q, -c + 0.1 * k, 0
    q, k, v, do = [t.to(BF).cuda() for t in (q, k, v, do)]
    grads = []
    for n in (L, whole):
        x = [t[:, :n].contiguous() for t in (q, k, v)]
        o, lse = api.attention_fwd(*x, causal=True)
        assert lse.max() < -89
        grads.append((o, lse) + api.attention_bwd(*x, o, lse, do[:, :n].contiguous(), causal=True))
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), *grads):
        assert torch.equal(a, b[:, :L]), name


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("lq", [21, 32, 64, 90])
def test_rows_past_the_end(dtype, D, lq):
    """A key of -infinity that every query scores -infinity has the probability
    0, as one of -1e30 has: the same o, lse, dk and dv, its own among them."""
    g = torch.Generator().manual_seed(D + lq)
    q, k, v, do = [torch.randn((2, n, h, D), generator=g) for n, h in ((lq, 6), (75, 2), (75, 2), (lq, 6))]
    q[..., 0] = q[..., 0].abs() + 0.5
    out = []
    for hidden in (-1e30, -float("inf")):
        k[:, 30, :, 0] = hidden
        x = [t.to(dtype).cuda() for t in (q, k, v, do)]
        o, lse = api.attention_fwd(*x[:3])
        out.append((o, lse) + api.attention_bwd(*x[:3], o, lse, x[3])[1:])
    for name, a, b in zip(("o", "lse", "dk", "dv"), *out):
        assert torch.equal(a, b), name
        if name[0] == "d":
            assert torch.all(b[:, 30] == 0), name
