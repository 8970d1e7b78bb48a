"""Host-side checks of the microscaled 4-bit operators and the experts' order
(no GPU): every function that include/bconv_mx4.h declares is exported and
bound, arguments are refused with the documented codes before anything is
launched, and the references hold the format's invariants."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import mx4_reference as ref
import popcount_convolution_amd as pca
from popcount_convolution_amd import _binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, WORKSPACE = pca.BCONV_ERR_INVALID_ARGUMENT, pca.BCONV_ERR_WORKSPACE
F32, BF16 = pca.BCONV_F32, pca.BCONV_BF16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_binding.LIB_PATH):
        from popcount_convolution_amd import _build
        _build.build()
    return pca.load_library()


def test_header_symbols_exported(lib):
    text = open(os.path.join(ROOT, "include", "bconv_mx4.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(bconv_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 10, names
    raw = ctypes.CDLL(_binding.LIB_PATH)
    assert not [n for n in names if not hasattr(raw, n)]
    assert not [n for n in names if not getattr(lib, n).argtypes]


def refused(f, *args, status=INVALID, text=None):
    with pytest.raises(pca.BconvError) as e:
        f(*args)
    assert e.value.status == status, e.value
    if text:
        assert text in str(e.value), e.value


# Addresses that are never touched: a call with a bad argument ends before a launch.
X, C, S, V = 1 << 20, 2 << 20, 3 << 20, 4 << 20


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(cols=0), dict(cols=(1 << 20) + 1), dict(dtype=3), dict(dtype=-1), dict(ldx=99), dict(ldx=(1 << 30) + 1),
    dict(x=None), dict(codes=None), dict(scales=None), dict(x=X + 1), dict(codes=C + 8), dict(scales=S + 4), dict(values=V + 1),
    dict(codes=X), dict(scales=X), dict(values=X), dict(values=C), dict(scales=C)])
def test_quantize_refuses(lib, change):
    a = dict(stream=None, rows=4, cols=100, dtype=BF16, x=X, ldx=100, codes=C, scales=S, values=V)
    a.update(change)
    refused(pca.bconv_mx4_quantize, *a.values())


def test_empty_calls(lib):
    pca.bconv_mx4_quantize(None, 0, 100, BF16, None, 100, None, None)
    pca.bconv_expert_gather(None, 0, 2, 10, BF16, None, 10, None, None, None)
    pca.bconv_expert_combine(None, 0, 2, 10, BF16, None, 10, None, F32, None, None)
    pca.bconv_expert_combine_backward(None, 0, 2, 10, BF16, None, 10, None, 10, None, None, F32, None, None)
    pca.bconv_mx4_linear_destroy(None)


def test_create_refuses(lib):
    for args in ((0, 32, 4), (1025, 32, 4), (1, 0, 4), (1, 32, 0), (1, (1 << 20) + 1, 4), (1, 32, (1 << 20) + 1),
                 (1, 1 << 20, 1 << 19), (1024, 1 << 15, 1 << 14)):
        refused(pca.bconv_mx4_linear_create, *args, None, C, S)
    refused(pca.bconv_mx4_linear_create, 1, 32, 4, None, None, S)
    refused(pca.bconv_mx4_linear_create, 1, 32, 4, None, C, None)
    refused(pca.bconv_mx4_linear_create, 1, 32, 4, None, C, S, V + 2)
    d = _binding.bconv_mx4_linear_desc_t(1, 32, 4)
    assert lib.bconv_mx4_linear_create(d, None, C, S, None, None) == INVALID
    h = ctypes.c_void_p()
    assert lib.bconv_mx4_linear_create(None, None, C, S, None, ctypes.byref(h)) == INVALID
    args = pca.bconv_mx4_rows_t()
    refused(pca.bconv_mx4_linear_forward, None, None, args)
    refused(pca.bconv_mx4_linear_workspace_size, None, args)


@pytest.mark.parametrize("change", [
    dict(pairs=-1), dict(pairs=(1 << 27) + 1), dict(experts=0), dict(experts=1025), dict(id_bytes=2), dict(ids=None), dict(offsets=None),
    dict(order=None), dict(position=None), dict(ids=X + 2), dict(offsets=C + 2), dict(order=S + 1), dict(position=V + 3),
    dict(order=X), dict(position=S), dict(offsets=S), dict(position=C)])
def test_sort_refuses(lib, change):
    a = dict(stream=None, pairs=100, experts=8, id_bytes=4, ids=X, offsets=C, order=S, position=V)
    a.update(change)
    refused(pca.bconv_expert_sort, *a.values())


def test_sort_workspace(lib):
    assert pca.bconv_expert_sort_workspace_size(8192, 64) == 0
    need = pca.bconv_expert_sort_workspace_size(100000, 64)
    assert need > 0
    refused(pca.bconv_expert_sort, None, 100000, 64, 8, X, C, S, V, None, 0, status=WORKSPACE)
    refused(pca.bconv_expert_sort, None, 100000, 64, 8, X, C, S, V, 5 << 20, need - 1, status=WORKSPACE)
    refused(pca.bconv_expert_sort, None, 100000, 64, 8, X, C, S, V, (5 << 20) + 4, need)
    refused(pca.bconv_expert_sort, None, 100000, 64, 8, X, C, S, V, S, need)
    refused(pca.bconv_expert_sort_workspace_size, -1, 8)


COMMON = [dict(tokens=-1), dict(choices=0), dict(tokens=1 << 20, choices=1 << 8), dict(width=0), dict(width=(1 << 20) + 1),
          dict(dtype=7), dict(position=None), dict(position=V + 2)]


@pytest.mark.parametrize("change", COMMON + [
    dict(ldx=9), dict(ldx=(1 << 30) + 1), dict(x=None), dict(order=None), dict(rows=None), dict(x=X + 1), dict(rows=C + 1),
    dict(order=S + 1), dict(rows=X), dict(rows=S), dict(rows=V)])
def test_gather_refuses(lib, change):
    a = dict(stream=None, tokens=5, choices=2, width=10, dtype=BF16, x=X, ldx=10, order=S, position=V, rows=C)
    a.update(change)
    refused(pca.bconv_expert_gather, *a.values())


@pytest.mark.parametrize("change", COMMON + [
    dict(ldr=9), dict(rows=None), dict(y=None), dict(rows=X + 1), dict(y=C + 1), dict(weight_dtype=3), dict(weights=S + 2),
    dict(y=X), dict(y=V), dict(y=S)])
def test_combine_refuses(lib, change):
    a = dict(stream=None, tokens=5, choices=2, width=10, dtype=BF16, rows=X, ldr=10, position=V, weight_dtype=F32, weights=S, y=C)
    a.update(change)
    refused(pca.bconv_expert_combine, *a.values())


@pytest.mark.parametrize("change", COMMON + [
    dict(ldd=9), dict(ldr=9), dict(dy=None), dict(rows=None), dict(order=None), dict(d_rows=None), dict(dy=X + 1), dict(rows=C + 1),
    dict(weight_dtype=3), dict(weights=(6 << 20) + 2), dict(d_weights=(8 << 20) + 1), dict(d_rows=X), dict(d_rows=C), dict(d_rows=S),
    dict(d_rows=V), dict(d_weights=X), dict(d_weights=6 << 20), dict(d_weights=7 << 20)])
def test_combine_backward_refuses(lib, change):
    a = dict(stream=None, tokens=5, choices=2, width=10, dtype=BF16, dy=X, ldd=10, rows=C, ldr=10, order=S, position=V,
             weight_dtype=F32, weights=6 << 20, d_rows=7 << 20, d_weights=8 << 20)
    a.update(change)
    refused(pca.bconv_expert_combine_backward, *a.values())


# ------------------------------------------------------------ torch wrappers

def test_wrappers_refuse_host_tensors(lib):
    x, ids = torch.zeros((4, 64)), torch.zeros((4, 2), dtype=torch.int64)
    for f in (lambda: pca.mx4_quantize(x), lambda: pca.sort_by_expert(ids, 4)):
        with pytest.raises(ValueError, match="device"):
            f()


@pytest.mark.parametrize("bad,match", [
    (np.zeros((2, 4)), "torch tensor"), (torch.zeros((2, 4), dtype=torch.int32), "dtype"), (torch.zeros(()), "does not end"),
    (torch.zeros((2, 0)), "does not end"), (torch.zeros((4, 8)).t(), "strides")])
def test_quantize_wrapper_refuses(lib, bad, match):
    with pytest.raises(ValueError, match=match):
        pca.mx4_quantize(bad)


@pytest.mark.parametrize("bad,experts,match", [
    ([[1]], 4, "torch tensor"), (torch.zeros((4, 2)), 4, "int32 or int64"), (torch.zeros(4, dtype=torch.int32), 4, "tokens, choices"),
    (torch.zeros((4, 0), dtype=torch.int32), 4, "tokens, choices"), (torch.zeros((2, 4), dtype=torch.int32).t(), 4, "contiguous")])
def test_sort_wrapper_refuses(lib, bad, experts, match):
    with pytest.raises(ValueError, match=match):
        pca.sort_by_expert(bad, experts)


def host_order(tokens=4, choices=2, experts=3):
    """An order whose tensors are on the host: wrappers look at shapes and types first."""
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    o = pca.ExpertOrder.__new__(pca.ExpertOrder)
    return o._set(ints(experts + 1), ints(tokens * choices), ints(tokens, choices), experts)


def test_order_tensors_are_checked(lib):
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = [ints(4), ints(8), ints(4, 2)]
    with pytest.raises(ValueError, match="device"):
        pca.ExpertOrder(*good, 3)
    for i, bad, match in ((0, ints(3), "offsets: shape"), (1, ints(7), "order: shape"), (2, ints(8), "position: shape"),
                          (1, ints(8).long(), "dtype"), (2, ints(2, 4).t(), "contiguous|device")):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError, match=match if i != 1 and i != 2 else match + "|device"):
            pca.ExpertOrder(*args, 3)


def test_order_refuses(lib):
    o = host_order()
    x, rows, w = torch.zeros((4, 10)), torch.zeros((8, 10)), torch.zeros((4, 2))
    for f, match in ((lambda: o.gather(rows), "not \\(4"), (lambda: o.combine(x, w), "not \\(8"),
                     (lambda: o.gather(x.to(torch.int32)), "dtype"), (lambda: o.gather(x[:, :0]), "1 to"),
                     (lambda: o.gather(x), "device"), (lambda: o.combine(rows), "device"),
                     (lambda: o.gather(torch.zeros((10, 4)).t()), "device")):
        with pytest.raises(ValueError, match=match):
            f()


# ---------------------------------------------------------------- references

def test_reference_format():
    """Values on the grid are kept, ties go to the even code, the largest of a
    block picks the power of two, and packing is undone."""
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6] * 4)[None] * np.array([1, -1] * 16)
    codes, scales, values = ref.quantise(grid)
    assert scales[0, 0] == 127 and np.array_equal(values, grid) and not codes[0, 16:].any() and not scales[0, 1:].any()
    ties = np.zeros((1, 32))
    ties[0, :9] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7]
    assert ref.quantise(ties)[2][0, :9].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 6]
    rng = np.random.default_rng(0)
    x = rng.normal(0, 1, (5, 300)) * 2.0 ** rng.integers(-20, 20, (5, 1))
    codes, scales, values = ref.quantise(x)
    assert codes.shape == (5, 256) and scales.shape == (5, 16)
    assert np.array_equal(ref.dense(codes, scales, 300), values)
    again = ref.quantise(values)
    # a block whose largest became less than 4 steps has another power of two; its values stay
    assert np.array_equal(again[2], values)
    # half a step of the upper part, 2 of 8 where the largest saturates
    top = np.abs(np.pad(x, ((0, 0), (0, 20))).reshape(5, 10, 32)).max(-1).repeat(32, 1)[:, :300]
    assert (np.abs(values - x) <= top / 4).all()


def test_reference_special():
    x = np.zeros((1, 96))
    x[0, 3], x[0, 40], x[0, 64] = np.nan, -np.inf, -0.0
    codes, scales, values = ref.quantise(x)
    assert scales[0, :3].tolist() == [255, 255, 0] and np.isnan(values[0, :64]).all() and not codes[0, :32].any()
    assert codes[0, 32] == 8 and np.signbit(values[0, 64])


def test_reference_order():
    offsets, order, position = ref.expert_order(np.array([[1, 0], [5, 1], [-1, 1]]), 3)
    assert offsets.tolist() == [0, 1, 4, 4] and order.tolist() == [1, 0, 3, 5, -1, -1]
    assert position.tolist() == [[1, 0], [-1, 2], [-1, 3]]
