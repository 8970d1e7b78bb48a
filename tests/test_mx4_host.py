"""Calls of the microscaled operators and experts' orders that must be refused on
the host, shown without a GPU: tensors that exist as shapes, strides and devices
alone stand for ones that would not fit, or would live on another GPU."""

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import popcount_convolution_amd as pca


def fake(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda:0")


def i32(*shape):
    return fake(*shape, dtype=torch.int32)


# A C call's numbers of 32 bits would be the low halves of these: too few rows would be moved.
@pytest.mark.parametrize("tokens,choices", [(2 ** 32 + 5, 1), (2 ** 16, 2 ** 16), (1, 2 ** 32 + 3), (2 ** 27 + 1, 1), (2 ** 24, 9)])
def test_order_refuses_more_pairs_than_a_sort(tokens, choices):
    with FakeTensorMode(), pytest.raises(ValueError, match=f"position: {tokens * choices} pairs are more than 2\\^27"):
        pca.ExpertOrder(i32(4), i32(tokens * choices), i32(tokens, choices), 3)


def test_order_takes_as_many_pairs_as_a_sort():
    with FakeTensorMode():
        o = pca.ExpertOrder(i32(4), i32(2 ** 27), i32(2 ** 24, 8), 3)
    assert (o.tokens, o.choices, o.experts) == (2 ** 24, 8, 3)


def layer(cls):
    made = object.__new__(cls)
    made.handle = None
    return made


def test_workspace_bytes_refuses():
    linear, experts = layer(pca.MX4Linear), layer(pca.MX4Experts)
    for f, match in ((lambda: linear.workspace_bytes(2 ** 32 + 1, torch.float32), "rows: .* is not a 32-bit number"),
                     (lambda: linear.workspace_bytes(1, torch.float64), "dtype"),
                     (lambda: experts.workspace_bytes(2 ** 32 + 1, 1, torch.float32), "tokens: .* is not a 32-bit number"),
                     (lambda: experts.workspace_bytes(2 ** 20, 2 ** 12 + 1, torch.float32), "rows: .* is not a 32-bit number"),
                     (lambda: experts.workspace_bytes(5, 0, torch.float32), "choices: 0"),
                     (lambda: experts.workspace_bytes(5, 2 ** 32 + 1, torch.float32), "choices"),
                     (lambda: experts.workspace_bytes(5, 2, torch.int32), "dtype")):
        with pytest.raises(ValueError, match=match):
            f()
    for f in (lambda: linear.workspace_bytes(1, torch.float32), lambda: experts.workspace_bytes(5, 2, torch.float32)):
        with pytest.raises(pca.BconvError, match="handle"):  # a closed layer
            f()
