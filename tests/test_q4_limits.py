"""Calls of the 4-bit operators that must be refused on the host, shown without a
GPU: tensors that exist as shapes, strides and devices alone stand for ones
that would not fit, or would live on another GPU."""

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import popcount_convolution_amd as pca


def fake(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda:0")


def q4_layer(n_in=64, n_out=32, device="cuda:0"):
    layer = object.__new__(pca.Q4Linear)
    layer.handle, layer.in_features, layer.out_features, layer.group = None, n_in, n_out, 32
    layer._needs, layer.device = {}, torch.device(device)
    return layer


def test_linear_refuses_another_gpu():
    """Rows on another GPU than the weights', with or without an output there."""
    with FakeTensorMode():
        for kw in ({}, {"out": fake(3, 32)}):
            with pytest.raises(ValueError, match="input: on cuda:0, not on cuda:1"):
                q4_layer(device="cuda:1").forward(fake(3, 64), **kw)


def test_convolution_refuses_another_gpu():
    """The same for the binary layers."""
    layer = object.__new__(pca.BinaryConvolution)
    layer.handle, layer.in_h, layer.in_w, layer.in_c, layer.device = None, 4, 4, 8, torch.device("cuda:1")
    with FakeTensorMode(), pytest.raises(ValueError, match="input: on cuda:0, the layer is on cuda:1"):
        layer.forward(fake(2, 4, 4, 8, dtype=torch.float32))
