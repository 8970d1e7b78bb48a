"""Microscaled 4-bit floats and layers of experts, torch-facing.

``mx4_quantize`` (rows to 4-bit floats with one power of two per 32 values),
``MX4Linear`` and ``MX4Experts`` (linear layers of such weights and inputs, one
or one for each expert), ``sort_by_expert`` and the ``ExpertOrder`` it returns
(tokens' rows into the experts' order and back with weights, and the gradients
of both).  As in ``q4``, torch provides device memory and the current stream;
every step runs in the kernels of ``libbconv.so`` (``include/bconv_mx4.h``
documents formats and formulas), tensors are checked before anything is
launched, and what a call allocates is allocated on the stream it launches on.
No call here is part of torch's autograd: results carry no gradient, also where
an input requires one.  Gradients are calls of their own, of the gather and the
combination; the products have none.
"""

from __future__ import annotations

from typing import NamedTuple

import numpy as np

from . import _binding as B
from . import q4 as _q4
from .q4 import (_INT32_MAX, _DTYPES, _dtype_code, _need_cuda, _need_dense, _need_int32, _need_tensor,
                 _need_workspace, _place, _row_stride)

BLOCK = 32   # values that share a power of two
_PAD = 256   # quantised rows are padded to a multiple of this
_MOST_PAIRS = 1 << 27  # (token, choice) pairs of an order


_torch = None  # the torch module, once a call needs it


def _load():
    global _torch
    _torch = _q4._torch or _q4._load_torch()
    return _torch


def _padded(cols: int) -> int:
    return -(-cols // _PAD) * _PAD


class MX4Tensor(NamedTuple):
    """Quantised rows: what ``mx4_quantize`` returns and linear layers take.  Layers'
    weights are held without the padding: ``codes[..., :ceil(cols / 2)]`` and
    ``scales[..., :ceil(cols / 32)]`` of quantised rows of weights."""
    codes: object   # uint8 [..., padded / 2], value 2 i of a row in the low half of byte i
    scales: object  # uint8 [..., padded / 32], exponent + 127 of a block of 32 values; 255: NaN
    cols: int       # values of a row; padded is that, rounded up to a multiple of 256 with zeros


def mx4_quantize(x, *, values: bool = False, stream=None):
    """``[..., cols]`` rows of float32, float16 or bfloat16 as an ``MX4Tensor``.
    With ``values`` returns ``(quantised, values)``, the tensor of x's shape and
    type that they stand for.  A 2-d x may have any row stride; others must be
    contiguous.  A block that holds a NaN or an infinity becomes NaN."""
    torch = _torch or _load()
    _need_tensor(x, "input")
    shape = x.shape
    if not shape or not 1 <= shape[-1] <= 1 << 20:
        raise ValueError(f"input: shape {tuple(shape)} does not end in 1 to {1 << 20} values")
    code = _dtype_code(x, "input")
    rows, ldx = _row_stride(x, "input")
    if rows > _INT32_MAX:
        _need_int32(rows, "input")
    _need_cuda(x, "input")
    *lead, cols = shape
    padded = _padded(cols)
    place, raw = _place(x.device, stream)
    with place:
        codes = x.new_empty((*lead, padded // 2), dtype=torch.uint8)
        scales = x.new_empty((*lead, padded // BLOCK), dtype=torch.uint8)
        dense = x.new_empty(shape) if values else None
        if rows:
            B.bconv_mx4_quantize(raw, rows, cols, code, x.data_ptr(), ldx, codes.data_ptr(), scales.data_ptr(),
                                 dense.data_ptr() if values else None)
    q = MX4Tensor(codes, scales, cols)
    return (q, dense) if values else q


class _MX4Layer:
    """Weights of one linear layer or one for each expert, and their product."""

    device = None  # where the weights are

    def _create(self, experts: int, in_features: int, out_features: int, lead: tuple, codes, scales, bias):
        self.handle = None
        self._needs: dict = {}  # workspace bytes by what decides them
        for name, value in (("experts", experts), ("in_features", in_features), ("out_features", out_features)):
            _need_int32(value, name)
            if value < 1:
                raise ValueError(f"{name}: {value} is not positive")
        torch = _torch or _load()
        self.in_features, self.out_features = in_features, out_features
        device = torch.device("cuda", torch.cuda.current_device())
        held = []
        for name, a, shape, dtype in (("codes", codes, (*lead, -(-in_features // 2)), torch.uint8),
                                      ("scales", scales, (*lead, -(-in_features // BLOCK)), torch.uint8),
                                      ("bias", bias, lead, torch.float32)):
            if a is None and name == "bias":
                held.append(None)
                continue
            t = a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))
            if t.dtype != dtype:
                raise ValueError(f"{name}: dtype {t.dtype} is not {dtype}")
            if tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
            if t.is_cuda and t.device != device:
                raise ValueError(f"{name}: on {t.device}, not on {device}")
            held.append(t.to(device).contiguous())
        raw = torch.cuda.current_stream(device).cuda_stream
        self.handle = B.bconv_mx4_linear_create(experts, in_features, out_features, raw, *[
            None if t is None else t.data_ptr() for t in held])
        self.device = device

    def _forward(self, x, dtype, out, workspace, stream, rows, out_lead, choices, offsets, order):
        """Product of checked rows: ``rows`` results of shape ``out_lead``."""
        torch = _torch
        device = self.device
        if type(x) is MX4Tensor:
            if dtype is None:
                dtype = torch.bfloat16 if out is None else out.dtype
            code = _DTYPES.get(dtype)
            if code is None:
                raise ValueError(f"dtype {dtype} is not one of torch.float32, torch.float16, torch.bfloat16")
            padded = _padded(self.in_features)
            shape = x.codes.shape[:-1]
            _need_dense(x.codes, "input codes", (*shape, padded // 2), torch.uint8, device)
            _need_dense(x.scales, "input scales", (*shape, padded // BLOCK), torch.uint8, device)
            x_rows = x.codes.numel() // (padded // 2)
            px, ldx, pc, ps = None, 0, x.codes.data_ptr(), x.scales.data_ptr()
        else:
            if dtype is not None and dtype is not x.dtype:
                raise ValueError(f"dtype {dtype}: results of {x.dtype} rows have their type")
            code = _dtype_code(x, "input")
            dtype = x.dtype
            x_rows, ldx = _row_stride(x, "input")
            if x.device != device:
                _need_cuda(x, "input", device)
            px, pc, ps = x.data_ptr(), None, None
        place, raw = _place(device, stream)
        with place:
            out_shape = (*out_lead, self.out_features)
            if out is None:
                out = torch.empty(out_shape, dtype=dtype, device=device) if px is None else x.new_empty(out_shape)
                ldy = self.out_features
            else:
                _need_tensor(out, "output")
                if tuple(out.shape) != out_shape:
                    raise ValueError(f"output: shape {tuple(out.shape)} != {out_shape}")
                if out.dtype != dtype:
                    raise ValueError(f"output: dtype {out.dtype} is not {dtype}")
                _need_cuda(out, "output", device)
                ldy = _row_stride(out, "output")[1]
            if rows == 0:
                return out
            args = B.bconv_mx4_rows_t(px, ldx, pc, ps, out.data_ptr(), ldy, x_rows, rows, code, choices, offsets,
                                      order)
            key = (rows, code, choices, px is None)
            need = self._needs.get(key)
            if need is None:
                need = B.bconv_mx4_linear_workspace_size(self.handle, args)
                if len(self._needs) >= 4096:
                    self._needs.clear()
                self._needs[key] = need
            if workspace is not None:
                _need_workspace(workspace, need, device)
            elif need:
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
            B.bconv_mx4_linear_forward(self.handle, raw, args, workspace.data_ptr() if need else None, need)
        return out

    def _workspace_bytes(self, rows: int, x_rows: int, choices: int, dtype, quantised: bool, experts: bool) -> int:
        if _torch is None:
            _load()
        code = _DTYPES.get(dtype)
        if code is None:
            raise ValueError(f"dtype {dtype} is not one of torch.float32, torch.float16, torch.bfloat16")
        _need_int32(rows, "rows")
        given = 16  # any address: of pointers, only whether they are there counts
        args = B.bconv_mx4_rows_t(None if quantised else given, 0, given if quantised else None,
                                  given if quantised else None, None, 0, x_rows, rows, code, choices,
                                  given if experts else None, given if choices else None)
        return B.bconv_mx4_linear_workspace_size(self.handle, args)

    def _input_shape(self, x):
        """Shape of the input's rows, without their values."""
        if type(x) is MX4Tensor:
            _need_tensor(x.codes, "input codes")
            _need_tensor(x.scales, "input scales")
            if x.cols != self.in_features or not x.codes.dim():
                raise ValueError(f"input: rows of {x.cols} values, not {self.in_features}")
            return x.codes.shape[:-1]
        _need_tensor(x, "input")
        shape = x.shape
        if not shape or shape[-1] != self.in_features:
            raise ValueError(f"input: shape {tuple(shape)} does not end in {self.in_features}")
        return shape[:-1]

    def close(self):
        if getattr(self, "handle", None):
            B.bconv_mx4_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MX4Linear(_MX4Layer):
    """A linear layer of microscaled 4-bit floats on the current GPU:
    ``y = Q(x) W^T + bias``, where Q is what ``mx4_quantize`` does to a row.

    ``codes``: uint8 ``[out_features, ceil(in_features/2)]``; ``scales``: uint8
    ``[out_features, ceil(in_features/32)]``; ``bias``: float32
    ``[out_features]`` or None; numpy arrays or tensors, copied.  ``forward`` sums in float32.
    """

    def __init__(self, *, in_features: int, out_features: int, codes, scales, bias=None):
        self._create(1, in_features, out_features, (out_features,), codes, scales, bias)

    def workspace_bytes(self, rows: int, dtype, *, quantised: bool = False) -> int:
        """Bytes of the workspace of a call with ``rows`` rows and results of
        ``dtype``, from an ``MX4Tensor`` if ``quantised``."""
        return self._workspace_bytes(rows, rows, 0, dtype, quantised, False)

    def forward(self, x, out=None, *, dtype=None, workspace=None, stream=None):
        """``[..., in_features]`` rows of float32, float16 or bfloat16 ->
        ``[..., out_features]`` of the same type; or an ``MX4Tensor`` of such rows
        -> ``dtype`` (out's, or bfloat16).  A 2-d x or out may have any row stride;
        others must be contiguous."""
        lead = self._input_shape(x)
        rows = 1
        for n in lead:
            rows *= n
        if rows > _INT32_MAX:
            _need_int32(rows, "input")
        return self._forward(x, dtype, out, workspace, stream, rows, lead, 0, None, None)


class ExpertOrder:
    """(token, choice) pairs in the order of their experts (2^27 at most), from
    ``sort_by_expert``, and what takes rows there and back.

    ``offsets``: int32 ``[experts + 1]``, where each expert's pairs start (the last:
    how many are not dropped); ``order``: int32 ``[tokens * choices]``, the pair
    token * choices + choice at each place, -1 behind the last; ``position``:
    int32 ``[tokens, choices]``, each pair's place, -1 where it is dropped."""

    def __init__(self, offsets, order, position, experts: int):
        torch = _torch or _load()
        _need_tensor(position, "position")
        if position.dim() != 2 or not position.shape[1]:
            raise ValueError(f"position: shape {tuple(position.shape)} is not (tokens, choices)")
        for name, t, shape in (("offsets", offsets, (experts + 1,)), ("order", order, (position.numel(),)),
                               ("position", position, position.shape)):
            _need_dense(t, name, shape, torch.int32, position.device)
        if position.numel() > _MOST_PAIRS:
            raise ValueError(f"position: {position.numel()} pairs are more than 2^27")
        self._set(offsets, order, position, experts)

    def _set(self, offsets, order, position, experts: int):
        self.offsets, self.order, self.position, self.experts = offsets, order, position, experts
        self.tokens, self.choices = position.shape
        self.device = position.device
        self._index = self.device.index  # None, as no tensor's get_device(), off the GPU
        return self

    def _rows(self, t, name: str, rows: int, dtype=None):
        """(width, row stride, dtype code) of a tensor ``[rows, width]``."""
        _need_tensor(t, name)
        shape = t.shape
        if len(shape) != 2 or shape[0] != rows or not 1 <= shape[1] <= 1 << 20:
            raise ValueError(f"{name}: shape {tuple(shape)} is not ({rows}, 1 to {1 << 20})")
        code = _dtype_code(t, name)
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name}: dtype {t.dtype} is not {dtype}")
        if t.get_device() != self._index:
            _need_cuda(t, name, self.device)
        width = shape[1]
        return width, width if t.is_contiguous() else _row_stride(t, name)[1], code

    def _weights(self, t):
        """Type code of the weights ``[tokens, choices]``."""
        _need_tensor(t, "weights")
        code = _dtype_code(t, "weights")
        if t.shape != self.position.shape or not t.is_contiguous() or t.get_device() != self._index:
            _need_dense(t, "weights", self.position.shape, t.dtype, self.device)
        return code

    def _result(self, out, name: str, shape, like):
        if out is None:
            return like.new_empty(shape)
        _need_dense(out, name, shape, like.dtype, self.device)
        return out

    def gather(self, x, out=None, stream=None):
        """Tokens' rows ``[tokens, width]`` -> ``[tokens * choices, width]`` in the
        experts' order; rows behind the last pair become 0."""
        width, ldx, code = self._rows(x, "x", self.tokens)
        place, raw = _place(self.device, stream)
        with place:
            out = self._result(out, "out", (self.tokens * self.choices, width), x)
            if self.tokens:
                B.bconv_expert_gather(raw, self.tokens, self.choices, width, code, x.data_ptr(), ldx,
                                      self.order.data_ptr(), self.position.data_ptr(), out.data_ptr())
        return out

    def gather_backward(self, d_rows, out=None, stream=None):
        """Gradient of ``gather``: that of its rows -> that of the tokens' rows.  (Of
        gathered rows that went through experts with gradients: those of
        ``MX4Experts`` have none, and take the tokens' rows themselves.)"""
        return self.combine(d_rows, None, out=out, stream=stream)

    def combine(self, rows, weights=None, out=None, stream=None):
        """Rows in the experts' order -> ``[tokens, width]``, the sum of each token's
        rows times its ``weights`` (``[tokens, choices]`` of float32, float16 or
        bfloat16; None for 1), without the dropped ones.  The result carries no
        gradient: a router learns from ``combine_backward``."""
        width, ldr, code = self._rows(rows, "rows", self.tokens * self.choices)
        weight_code = 0 if weights is None else self._weights(weights)
        place, raw = _place(self.device, stream)
        with place:
            out = self._result(out, "out", (self.tokens, width), rows)
            if self.tokens:
                B.bconv_expert_combine(raw, self.tokens, self.choices, width, code, rows.data_ptr(), ldr,
                                       self.position.data_ptr(), weight_code,
                                       None if weights is None else weights.data_ptr(), out.data_ptr())
        return out

    def combine_backward(self, dy, rows, weights=None, d_rows=None, d_weights=None, stream=None):
        """Gradient of ``combine``: ``(d_rows, d_weights)`` for the gradient ``dy``
        ``[tokens, width]`` of its result, ``d_weights`` None without ``weights``
        (``rows`` is not read then).  Rows behind the last pair and weights of
        dropped pairs have the gradient 0.  ``d_rows`` and ``d_weights`` may be given to be filled."""
        width, ldd, code = self._rows(dy, "dy", self.tokens)
        pairs = self.tokens * self.choices
        weight_code, ldr = 0, width
        if weights is not None:
            weight_code = self._weights(weights)
            row_width, ldr, _ = self._rows(rows, "rows", pairs, dy.dtype)
            if row_width != width:
                raise ValueError(f"rows: {row_width} values, dy has {width}")
        elif d_weights is not None:
            raise ValueError("d_weights: given without weights")
        place, raw = _place(self.device, stream)
        with place:
            d_rows = self._result(d_rows, "d_rows", (pairs, width), dy)
            if weights is not None:
                d_weights = self._result(d_weights, "d_weights", self.position.shape, weights)
            if self.tokens:
                B.bconv_expert_combine_backward(
                    raw, self.tokens, self.choices, width, code, dy.data_ptr(), ldd,
                    None if weights is None else rows.data_ptr(), ldr, self.order.data_ptr(), self.position.data_ptr(),
                    weight_code, None if weights is None else weights.data_ptr(), d_rows.data_ptr(),
                    None if weights is None else d_weights.data_ptr())
        return d_rows, d_weights


_sort_needs: dict = {}  # workspace bytes by (pairs, experts)


def sort_by_expert(expert_ids, experts: int, stream=None) -> ExpertOrder:
    """Sorts the pairs of ``expert_ids`` (int32 or int64 ``[tokens, choices]``, the
    experts that each token chose) by expert, those of an expert in their order.
    Pairs whose id is not in ``[0, experts)`` are dropped."""
    torch = _torch or _load()
    _need_tensor(expert_ids, "expert_ids")
    if expert_ids.dtype not in (torch.int32, torch.int64) or expert_ids.dim() != 2 or not expert_ids.shape[1]:
        raise ValueError(f"expert_ids: {expert_ids.dtype} of shape {tuple(expert_ids.shape)} is not int32 or int64 "
                         "(tokens, choices)")
    if not expert_ids.is_contiguous():
        raise ValueError("expert_ids: the tensor must be contiguous")
    _need_cuda(expert_ids, "expert_ids")
    if not 1 <= experts <= 1024:
        raise ValueError(f"experts: {experts} is not in [1, 1024]")
    device = expert_ids.device
    tokens, choices = expert_ids.shape
    pairs = tokens * choices
    if pairs > _INT32_MAX:
        _need_int32(pairs, "expert_ids")
    place, raw = _place(device, stream)
    with place:
        # one allocation: offsets, order, positions
        flat = torch.empty(experts + 1 + 2 * pairs, dtype=torch.int32, device=device)
        offsets, order, position = flat.split_with_sizes((experts + 1, pairs, pairs))
        need = _sort_needs.get((pairs, experts))
        if need is None:
            need = B.bconv_expert_sort_workspace_size(pairs, experts)
            if len(_sort_needs) >= 4096:
                _sort_needs.clear()
            _sort_needs[pairs, experts] = need
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        base = flat.data_ptr()
        B.bconv_expert_sort(raw, pairs, experts, expert_ids.element_size(), expert_ids.data_ptr(), base,
                            base + 4 * (experts + 1), base + 4 * (experts + 1 + pairs), workspace, need)
    return ExpertOrder.__new__(ExpertOrder)._set(offsets, order, position.view(tokens, choices), experts)


class MX4Experts(_MX4Layer):
    """Linear layers of microscaled 4-bit floats, one for each expert, on the
    current GPU, applied to the rows that chose it.

    ``codes``: uint8 ``[experts, out_features, ceil(in_features/2)]``; ``scales``:
    uint8 ``[experts, out_features, ceil(in_features/32)]``; ``bias``: float32
    ``[experts, out_features]`` or None; numpy arrays or tensors, copied."""

    def __init__(self, *, experts: int, in_features: int, out_features: int, codes, scales, bias=None):
        self.experts = experts
        self._create(experts, in_features, out_features, (experts, out_features), codes, scales, bias)

    def workspace_bytes(self, tokens: int, choices: int, dtype, *, in_order: bool = False, quantised: bool = False) -> int:
        """Bytes of the workspace of a call with an order of ``tokens`` times
        ``choices`` pairs and results of ``dtype``, from an ``MX4Tensor`` if ``quantised``."""
        _need_int32(tokens, "tokens")
        if not 1 <= choices <= _INT32_MAX:
            raise ValueError(f"choices: {choices} is not in [1, {_INT32_MAX}]")
        rows = tokens * choices
        return self._workspace_bytes(rows, rows if in_order else tokens, 0 if in_order else choices, dtype, quantised, True)

    def forward(self, x, order: ExpertOrder, out=None, *, in_order: bool = False, dtype=None, workspace=None,
                stream=None):
        """``[tokens, in_features]`` rows (or, ``in_order``, ``[tokens * choices,
        in_features]`` rows in the experts' order, such as another layer's results) ->
        ``[tokens * choices, out_features]`` rows in the experts' order, of x's type;
        an ``MX4Tensor`` of such rows -> ``dtype`` (out's, or bfloat16).  Rows
        behind the last pair become 0.  A row stride is free for x and out."""
        lead = self._input_shape(x)
        if not isinstance(order, ExpertOrder):
            raise ValueError(f"order: an ExpertOrder is required, got {type(order).__name__}")
        if order.experts != self.experts:
            raise ValueError(f"order: of {order.experts} experts, the layer has {self.experts}")
        if order.device != self.device:
            raise ValueError(f"order: on {order.device}, not on {self.device}")
        rows = order.tokens * order.choices
        want = (rows,) if in_order else (order.tokens,)
        if tuple(lead) != want:
            raise ValueError(f"input: {tuple(lead)} rows, the order needs {want}")
        return self._forward(x, dtype, out, workspace, stream, rows, (rows,), 0 if in_order else order.choices,
                             order.offsets.data_ptr(), None if in_order else order.order.data_ptr())
