"""Which views attention takes, on the host: the token stride that the torch
wrapper passes across the ABI (0 there means packed), and the ABI's own bounds.
"""
import pytest
import torch

from gated_deltanet_scan_amd import api


@pytest.mark.parametrize("one,shape", [
    ((1, 1, 4, 64), (8, 1, 4, 64)), ((1, 1, 1, 4, 64), (8, 1, 1, 4, 64)),        # single tokens
    ((1, 5, 4, 64), (8, 5, 4, 64)), ((1, 3, 5, 4, 64), (8, 3, 5, 4, 64)),        # whole sequences
    ((1, 1, 4, 64), (1, 5, 4, 64)), ((2, 1, 4, 64), (2, 5, 4, 64)), ((1, 4, 64), (6, 4, 64)),   # along the tokens
    ((2, 5, 1, 64), (2, 5, 4, 64)), ((2, 1, 1, 64), (2, 1, 4, 64)),              # along the heads
])
def test_broadcast_inputs_are_refused(one, shape):
    t = torch.zeros(one).expand(shape)
    with pytest.raises(ValueError, match="evenly spaced tokens"):
        api._token_strides(t, "q")


def test_overlapping_single_tokens_are_refused():
    t = torch.zeros(4096).as_strided((8, 1, 4, 64), (128, 256, 64, 1))            # tokens share half their heads
    with pytest.raises(ValueError, match="evenly spaced tokens"):
        api._token_strides(t, "q")


@pytest.mark.parametrize("shape", [(8, 1, 4, 64), (8, 1, 1, 4, 64), (2, 5, 4, 64), (2, 3, 5, 4, 64), (6, 4, 64)])
def test_views_that_are_taken(shape):
    H, D = shape[-2:]
    assert api._token_strides(torch.zeros(shape), "q") == (H * D, 0)
    fused = torch.zeros(shape[:-2] + (3 * H, D))[..., H:2 * H, :]
    assert api._token_strides(fused, "q") == (3 * H * D, 0)
    if len(shape) == 4:
        cache = torch.zeros((shape[0], 9) + shape[2:])[:, :shape[1]]
        want = (9 * H * D, 0) if shape[1] == 1 else (H * D, 9)
        assert api._token_strides(cache, "k") == want
