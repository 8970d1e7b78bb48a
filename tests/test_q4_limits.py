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


# ------------------------------------- numbers that an int32 does not hold
# (a C call's would be their low 32 bits: too few rows computed, or another stride)

def i32(*shape):
    return fake(*shape, dtype=torch.int32)


def test_linear_refuses_rows_past_32_bits():
    with FakeTensorMode():
        for x in (fake(2 ** 32 + 5, 1), fake(2 ** 16, 2 ** 15, 1)):
            with pytest.raises(ValueError, match="input: .* is not a 32-bit number"):
                q4_layer(n_in=1).forward(x)
    with pytest.raises(ValueError, match="rows: .* is not a 32-bit number"):
        q4_layer().workspace_bytes(2 ** 32 + 1, torch.float32)
    with pytest.raises(ValueError, match="dtype"):
        q4_layer().workspace_bytes(1, torch.float64)
    for sizes in ({"in_features": 2 ** 32 + 32, "out_features": 1}, {"in_features": 32, "out_features": 2 ** 32 + 1}):
        with pytest.raises(ValueError, match="features: .* is not a 32-bit number"):
            pca.Q4Linear(**sizes, weight_words=None, scales=None)


def cache():
    c = object.__new__(pca.KV4Cache)
    c.kv_heads, c.head_dim, c.block_size, c.device, c._needs = 1, 8, 16, torch.device("cuda:0"), {}
    return c


def test_cache_refuses_tokens_past_32_bits():
    many = 2 ** 32 + 5
    with FakeTensorMode():
        with pytest.raises(ValueError, match="k: .* is not a 32-bit number"):
            row = fake(1, 1, 8)
            cache().append(row.expand(many, 1, 8), row.expand(many, 1, 8), i32(many))
        with pytest.raises(ValueError, match="q: .* is not a 32-bit number"):
            cache().attention(fake(1, 1, 8).expand(many, 1, 8), i32(1, 2), i32(1))
        with pytest.raises(ValueError, match="block_table: .* is not a 32-bit number"):
            cache().attention(fake(2, 1, 8), i32(2, many)[:, :4], i32(2))
        with pytest.raises(ValueError, match="block_table: .* is not a 32-bit number"):
            cache().attention(fake(2, 1, 8), i32(1, many), i32(1))


def test_block_tables_refuse_numbers_past_32_bits():
    many = 2 ** 32 + 5
    with FakeTensorMode():
        for table, free, name in ((i32(2, many)[:, :4], i32(3), "block_table"), (i32(many, 1), i32(3), "block_table"),
                                  (i32(2, 4), i32(many), "free_blocks")):
            n = table.shape[0]
            with pytest.raises(ValueError, match=name + ": .* is not a 32-bit number"):
                pca.build_block_tables(table, i32(n), i32(n), free, i32(1), block_size=16, tokens=1)


def test_block_tables_refuse_results_over_inputs():
    """Each result one element into each input, and at its last."""
    at = dict(table=0x1000, ctx=0x2000, new=0x3000, free=0x4000, head=0x5000)
    size = dict(table=12, ctx=3, new=3, free=5, head=1)
    out = dict(lens=0x6000, start=0x7000, slots=0x8000, positions=0x9000, out_head=0xa000)

    def call(**kw):
        a = {**at, **out, **kw}
        pca.bconv_block_tables(None, 3, 16, a["table"], 4, 4, a["ctx"], a["new"], a["free"], 5, a["head"],
                               a["out_head"], 2, a["slots"], a["positions"], a["start"], a["lens"])

    for name in out:
        for where, base in at.items():
            for k in (0, size[where] - 1):
                with pytest.raises(pca.BconvError, match="overlaps"):
                    call(**{name: base + 4 * k})
