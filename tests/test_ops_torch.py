"""Calls that the torch side of the operators around the scan refuses, on the
host.
"""
import types

import pytest
import torch

from gated_deltanet_scan_amd import api, autograd


def test_positions_take_no_gradient():
    """rotary() has gradients to q and k; positions that ask for one would
    silently go without."""
    q = torch.zeros(4, 2, 64, requires_grad=True)
    pos = torch.zeros(4, 1, requires_grad=True)
    with pytest.raises(ValueError, match="positions"):
        autograd.rotary(q, None, pos, axes=(64,))
    for p in (pos.detach(), pos):                         # taken: the refusal is that of host tensors
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
            autograd.rotary(q, None, p, axes=(64,))
    with pytest.raises(ValueError, match="device tensor"):
        autograd.rotary(q, None, pos.detach(), axes=(64,))


def test_stream_of_another_device():
    """A launch there would read the tensors' addresses on the wrong device."""
    other = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        api._launch(other, torch.device("cuda:0"))
