"""4-bit operators of a language model's decoding step, torch-facing.

``Q4Linear`` (linear layers with 4-bit weights and group scales), ``KV4Cache``
(a paged cache of keys and values in 4 bits, with ``append`` and
``attention``) and ``build_block_tables`` (block tables and slot maps from
request lengths).  As in the rest of the package, torch provides device memory
and the current stream; every step runs in the kernels of ``libbconv.so``
(``include/bconv_q4.h`` documents formats and formulas).  Tensors are checked
before anything is launched, since the C side trusts the sizes it is given, and
what a call allocates is allocated on the stream it launches on.
"""

from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional

import numpy as np

from . import _binding as B

_torch = None      # the torch module, once a call needs it
_DTYPES: dict = {}  # torch dtype -> bconv_dtype_t


def _load_torch():
    global _torch, _raw_stream, _current_device
    import torch
    _DTYPES.update({torch.float32: B.BCONV_F32, torch.float16: B.BCONV_F16, torch.bfloat16: B.BCONV_BF16})
    # the current stream's handle without a Stream object around it, where torch has that
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)
    # the current device's index, without the check that CUDA is initialised (a device tensor is in hand)
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _torch = torch
    return torch


def _dtype_code(t, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: dtype {t.dtype} is not one of torch.float32, torch.float16, torch.bfloat16")
    return code


def _need_tensor(t, name: str) -> None:
    if not isinstance(t, _torch.Tensor):
        raise ValueError(f"{name}: a torch tensor is required, got {type(t).__name__}")


def _need_cuda(t, name: str, device=None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA (HIP) device tensor is required, got device {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, not on {device}")


def _need_dense(t, name: str, shape, dtype, device) -> None:
    """A contiguous device tensor of exactly ``shape`` and ``dtype``."""
    _need_tensor(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} is not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: the tensor must be contiguous")
    _need_cuda(t, name, device)


def _need_ints(t, name: str, count: int, device) -> None:
    """A contiguous int32 device tensor [count]."""
    if not (isinstance(t, _torch.Tensor) and t.dtype is _torch.int32 and t.dim() == 1 and t.numel() == count
            and t.is_contiguous() and t.is_cuda and t.get_device() == device.index):
        _need_dense(t, name, (count,), _torch.int32, device)


_INT32_MAX = 0x7fffffff


def _need_int32(value, name: str) -> None:
    """A number that the C side's int32 holds (ctypes would wrap others).  Sizes
    of tensors, which are not negative, are compared in place: a call of this costs
    a decoding step's calls 0.1 us each."""
    if not -0x80000000 <= value <= _INT32_MAX:
        raise ValueError(f"{name}: {value} is not a 32-bit number")


def _need_rows(t, name: str, heads: int, dim: int) -> int:
    """[tokens, heads, dim] with contiguous channels; token and head strides
    are free.  Returns the tokens."""
    _need_tensor(t, name)
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name}: shape {tuple(shape)} is not (tokens, {heads}, {dim})")
    if t.stride(2) != 1 and dim > 1:
        raise ValueError(f"{name}: channels must be contiguous (stride {t.stride(2)})")
    if shape[0] > _INT32_MAX:
        _need_int32(shape[0], name)
    return shape[0]


def _need_table(t) -> tuple:
    """(requests, width, row stride) of a block table."""
    _need_tensor(t, "block_table")
    if t.dtype != _torch.int32 or t.dim() != 2:
        raise ValueError(f"block_table: {t.dtype} of shape {tuple(t.shape)} is not int32 (requests, width)")
    requests, width = t.shape
    stride = t.stride()
    if width > 1 and stride[1] != 1 or requests > 1 and stride[0] < width:
        raise ValueError("block_table: rows must be contiguous and must not overlap")
    step = stride[0] if requests > 1 else max(width, 1)
    if requests > _INT32_MAX or step > _INT32_MAX:  # the step is no less than the width
        _need_int32(max(requests, step), "block_table")
    return requests, width, step


def _need_workspace(ws, need: int, device) -> None:
    _need_tensor(ws, "workspace")
    if not ws.is_contiguous():
        raise ValueError("workspace: the tensor must be contiguous")
    _need_cuda(ws, "workspace", device)
    have = ws.numel() * ws.element_size()
    if have < need:
        raise ValueError(f"workspace: {have} bytes given, {need} needed")


@contextlib.contextmanager
def _on(device, stream):
    with _torch.cuda.device(device), _torch.cuda.stream(stream):
        yield


_STAY = contextlib.nullcontext()


def _place(device, stream):
    """(context to allocate and launch in, raw stream): nothing to enter when
    the call goes to the current device's current stream."""
    if stream is None:
        if device.index == _current_device():
            return _STAY, _raw_stream(device.index)
        stream = _torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream: on {stream.device}, the tensors are on {device}")
    return _on(device, stream), stream.cuda_stream


def pack_codes(codes) -> np.ndarray:
    """[out, in] array of codes 0..15 as the uint32 words of ``Q4Linear``:
    input i of an output at bits 4 * (i % 8) of word i // 8."""
    c = np.asarray(codes)
    if c.ndim != 2:
        raise ValueError(f"codes: {c.ndim} dimensions, 2 needed")
    if c.size and (c.min() < 0 or c.max() > 15):
        raise ValueError("codes: values must be in [0, 15]")
    n, k = c.shape
    padded = np.zeros((n, -(-k // 8) * 8), np.uint32)
    padded[:, :k] = c
    return (padded.reshape(n, -1, 8) << (4 * np.arange(8, dtype=np.uint32))).sum(-1, dtype=np.uint32)


class Q4Linear:
    """A linear layer with 4-bit weights and group scales on the current GPU:
    ``y = x W^T + bias`` with ``W = scale * (code - zero)`` per group of inputs.

    ``weight_words``: host uint32 ``[out_features, ceil(in_features/8)]`` (see
    ``pack_codes``); ``scales``: host float16 ``[out_features,
    ceil(in_features/group)]``; ``zeros``: host uint8 of that shape, or None for
    8; ``bias``: host float32 ``[out_features]`` or None.  ``forward`` takes
    float32, float16 or bfloat16 rows on that GPU (``device``) and sums in float32.
    """

    device = None  # where the weights are

    def __init__(self, *, in_features: int, out_features: int, weight_words, scales, zeros=None, bias=None,
                 group: int = 128):
        self.handle = None
        self._needs: dict = {}  # workspace bytes by (rows, type)
        if group not in (32, 64, 128):
            raise ValueError(f"group: {group} is not 32, 64 or 128")
        _need_int32(in_features, "in_features")
        _need_int32(out_features, "out_features")
        groups = -(-in_features // group)
        for name, a, shape in (("weight_words", weight_words, (out_features, -(-in_features // 8))),
                               ("scales", scales, (out_features, groups)), ("zeros", zeros, (out_features, groups)),
                               ("bias", bias, (out_features,))):
            if a is not None and tuple(np.shape(a)) != shape:
                raise ValueError(f"{name}: shape {tuple(np.shape(a))} != {shape}")
        if np.asarray(weight_words).dtype != np.uint32:
            raise ValueError(f"weight_words: dtype {np.asarray(weight_words).dtype} is not uint32")
        if np.asarray(scales).dtype != np.float16:
            raise ValueError(f"scales: dtype {np.asarray(scales).dtype} is not float16")
        if zeros is not None and np.asarray(zeros).dtype != np.uint8:
            raise ValueError(f"zeros: dtype {np.asarray(zeros).dtype} is not uint8")
        self.in_features, self.out_features, self.group = in_features, out_features, group
        torch = _torch or _load_torch()
        self.handle = B.bconv_q4_linear_create(in_features, out_features, group, weight_words, scales, zeros, bias)
        self.device = torch.device("cuda", torch.cuda.current_device())

    def workspace_bytes(self, rows: int, dtype) -> int:
        if _torch is None:
            _load_torch()
        if dtype not in _DTYPES:
            raise ValueError(f"dtype {dtype} is not one of torch.float32, torch.float16, torch.bfloat16")
        _need_int32(rows, "rows")
        return B.bconv_q4_linear_workspace_size(self.handle, rows, _DTYPES[dtype])

    def forward(self, x, out=None, workspace=None, stream=None):
        """``[..., in_features]`` -> ``[..., out_features]`` of the same type.
        A 2-d x or out may have any row stride; others must be contiguous."""
        if _torch is None:
            _load_torch()
        _need_tensor(x, "input")
        shape = x.shape
        if not shape or shape[-1] != self.in_features:
            raise ValueError(f"input: shape {tuple(shape)} does not end in {self.in_features}")
        code = _dtype_code(x, "input")
        rows, ldx = _row_stride(x, "input")
        if rows > _INT32_MAX:
            _need_int32(rows, "input")
        device = x.device
        if device != self.device:
            _need_cuda(x, "input", self.device)
        place, raw = _place(device, stream)
        with place:
            out_shape = (*shape[:-1], self.out_features)
            if out is None:
                out = x.new_empty(out_shape)
                ldy = self.out_features
            else:
                _need_tensor(out, "output")
                if tuple(out.shape) != out_shape:
                    raise ValueError(f"output: shape {tuple(out.shape)} != {out_shape}")
                if out.dtype != x.dtype:
                    raise ValueError(f"output: dtype {out.dtype} is not {x.dtype}")
                _need_cuda(out, "output", device)
                ldy = _row_stride(out, "output")[1]
            if rows == 0:
                return out
            need = self._needs.get((rows, code))
            if need is None:
                need = self._needs[rows, code] = B.bconv_q4_linear_workspace_size(self.handle, rows, code)
            if workspace is not None:
                _need_workspace(workspace, need, device)
            elif need:
                workspace = _torch.empty(need, dtype=_torch.uint8, device=device)
            B.bconv_q4_linear_forward(self.handle, raw, rows, code, x.data_ptr(), ldx, out.data_ptr(), ldy,
                                      workspace.data_ptr() if need else None, need)
        return out

    def close(self):
        if getattr(self, "handle", None):
            B.bconv_q4_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _row_stride(t, name: str):
    """(rows, elements between rows) of a tensor whose last axis is contiguous."""
    width = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // width if width else 0), max(1, width)
    if t.dim() == 2 and (t.stride(1) == 1 or width == 1) and (t.stride(0) >= width or t.shape[0] == 1):
        return t.shape[0], max(t.stride(0), width)
    raise ValueError(f"{name}: strides {tuple(t.stride())}: only 2-d tensors with contiguous rows may be strided")


class KV4Cache:
    """Keys and values of a paged cache, 4 bits a channel with an fp16 step and
    midpoint per token, head and group of channels.

    ``pool`` holds ``num_blocks`` blocks of ``block_size`` tokens on ``device``
    (the current GPU by default), cleared at creation.
    """

    def __init__(self, num_blocks: int, block_size: int, kv_heads: int, head_dim: int, *, group: int = 64,
                 device=None):
        torch = _torch or _load_torch()
        for name, value in (("num_blocks", num_blocks), ("block_size", block_size), ("kv_heads", kv_heads),
                            ("head_dim", head_dim), ("group", group)):
            _need_int32(value, name)
        self.desc = B.bconv_kv4_desc_t(num_blocks, block_size, kv_heads, head_dim, group)
        self.layout = B.bconv_kv4_layout(self.desc)
        self.num_blocks, self.block_size, self.kv_heads = num_blocks, block_size, kv_heads
        self.head_dim, self.group = head_dim, group
        self.pool = torch.zeros(self.layout.pool_bytes, dtype=torch.uint8, device=device or "cuda")
        _need_cuda(self.pool, "device")
        self.device = self.pool.device
        self._needs: dict = {}  # workspace bytes of attention by its host arguments

    def append(self, k, v, slots, *, values: bool = False, k_out=None, v_out=None, stream=None):
        """Writes new rows ``[tokens, kv_heads, head_dim]`` at ``slots`` (int32
        ``[tokens]``, block * block_size + offset; slots outside the pool are
        skipped).  With ``values`` (or ``k_out`` / ``v_out``) returns the pair of
        dense tensors that the cache now stands for."""
        torch = _torch or _load_torch()
        heads, dim, device = self.kv_heads, self.head_dim, self.device
        tokens = _need_rows(k, "k", heads, dim)
        if _need_rows(v, "v", heads, dim) != tokens:
            raise ValueError(f"v: {v.shape[0]} tokens, k has {tokens}")
        code = _dtype_code(k, "k")
        if v.dtype != k.dtype:
            raise ValueError(f"v: dtype {v.dtype} is not {k.dtype}")
        _need_cuda(k, "k", device)
        _need_cuda(v, "v", device)
        _need_ints(slots, "slots", tokens, device)
        place, raw = _place(device, stream)
        with place:
            shape = (tokens, heads, dim)
            if k_out is not None:
                _need_dense(k_out, "k_out", shape, k.dtype, device)
            elif values:
                k_out = k.new_empty(shape)
            if v_out is not None:
                _need_dense(v_out, "v_out", shape, k.dtype, device)
            elif values:
                v_out = k.new_empty(shape)
            if tokens:
                B.bconv_kv4_append(self.desc, raw, self.pool.data_ptr(), tokens, code, k.data_ptr(), k.stride()[:2],
                                   v.data_ptr(), v.stride()[:2], slots.data_ptr(),
                                   None if k_out is None else k_out.data_ptr(),
                                   None if v_out is None else v_out.data_ptr())
        return (k_out, v_out) if k_out is not None or v_out is not None else None

    def attention(self, q, block_table, context_lens, *, q_start=None, max_q: Optional[int] = None,
                  max_context: int = 0, scale: Optional[float] = None, window: int = 0, out=None, lse=None,
                  workspace=None, stream=None):
        """``softmax(scale q K^T + mask) V`` for ``q`` ``[tokens, heads, head_dim]``.

        ``block_table``: int32 ``[requests, width]``; ``context_lens``: int32
        ``[requests]``, cached tokens with the new ones; ``q_start``: int32
        ``[requests + 1]`` prefix sums of the requests' queries, with ``max_q`` the
        most of one request (all tokens by default, which launches workgroups for
        that many in every request: give it where it is known), or None for the same
        number each.  ``max_context``
        bounds the context lengths (the table's width by default).  ``scale``
        defaults to ``head_dim ** -0.5``; ``window`` > 0 limits a query to that many
        last positions.  ``lse``: float32 ``[tokens, heads]`` to fill.  Rows of tokens
        that ``q_start`` gives to no request are not written."""
        torch = _torch or _load_torch()
        _need_tensor(q, "q")
        shape = q.shape
        if len(shape) != 3 or shape[1] % self.kv_heads or not shape[1]:
            raise ValueError(f"q: shape {tuple(shape)} is not (tokens, a multiple of {self.kv_heads}, "
                             f"{self.head_dim})")
        tokens, heads, dim = shape
        _need_rows(q, "q", heads, self.head_dim)
        code = _dtype_code(q, "q")
        device = self.device
        _need_cuda(q, "q", device)
        requests, width, stride = _need_table(block_table)
        _need_cuda(block_table, "block_table", device)
        _need_ints(context_lens, "context_lens", requests, device)
        if q_start is not None:
            _need_ints(q_start, "q_start", requests + 1, device)
            if max_q is None:
                max_q = max(1, tokens)
        else:
            if requests and tokens % requests:
                raise ValueError(f"q: {tokens} tokens are not a multiple of {requests} requests (pass q_start)")
            if max_q is None:
                max_q = max(1, tokens // requests if requests else 1)
        _need_int32(max_q, "max_q")
        _need_int32(max_context, "max_context")
        _need_int32(window, "window")
        place, raw = _place(device, stream)
        with place:
            if out is None:
                out = q.new_empty(shape)
            else:
                _need_dense(out, "out", shape, q.dtype, device)
            if lse is not None:
                _need_dense(lse, "lse", (tokens, heads), torch.float32, device)
            if not tokens or not requests:
                return out
            q_strides = q.stride()
            args = B.bconv_kv4_attention_t(
                self.pool.data_ptr(), q.data_ptr(), q_strides[0], q_strides[1], out.data_ptr(),
                None if lse is None else lse.data_ptr(), block_table.data_ptr(), context_lens.data_ptr(),
                None if q_start is None else q_start.data_ptr(), requests, tokens, max_q, heads, width, stride,
                max_context, window, code, dim ** -0.5 if scale is None else scale)
            key = (requests, tokens, max_q, heads, width, max_context, window, code, q_start is None)
            need = self._needs.get(key)
            if need is None:
                need = B.bconv_kv4_attention_workspace_size(self.desc, args)
                if len(self._needs) >= 4096:
                    self._needs.clear()
                self._needs[key] = need
            if workspace is not None:
                _need_workspace(workspace, need, device)
            elif need:
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
            B.bconv_kv4_attention(self.desc, raw, args, workspace.data_ptr() if need else None, need)
        return out


class BlockTables(NamedTuple):
    """What ``build_block_tables`` returns; every tensor int32."""
    slots: object         # [tokens] block * block_size + offset, -1 without a block
    positions: object     # [tokens] position in the request
    q_start: object       # [requests + 1] prefix sums of new_lens
    context_lens: object  # [requests] lengths with the new tokens
    free_head: object     # [1] first unused index of free_blocks


def build_block_tables(block_table, context_lens, new_lens, free_blocks, free_head, *, block_size: int, tokens: int,
                       stream=None) -> BlockTables:
    """Extends ``block_table`` (int32 ``[requests, width]``, in place) for
    ``new_lens`` more tokens a request, taking blocks from ``free_blocks`` at
    index ``free_head`` (int32 ``[1]``) on, and returns where the new tokens go.
    ``tokens``: entries of the slot map, at least the sum of ``new_lens`` (the
    rest is padded with -1).  All tensors are int32 on one device; ``free_head``
    of the result beyond ``free_blocks`` says that blocks were missing."""
    torch = _torch or _load_torch()
    requests, width, stride = _need_table(block_table)
    _need_cuda(block_table, "block_table")
    device = block_table.device
    _need_ints(context_lens, "context_lens", requests, device)
    _need_ints(new_lens, "new_lens", requests, device)
    _need_tensor(free_blocks, "free_blocks")
    free_count = free_blocks.numel()
    if free_count > _INT32_MAX:
        _need_int32(free_count, "free_blocks")
    _need_ints(free_blocks, "free_blocks", free_count, device)
    _need_ints(free_head, "free_head", 1, device)
    if tokens < 0:
        raise ValueError(f"tokens: {tokens} is negative")
    _need_int32(tokens, "tokens")
    _need_int32(block_size, "block_size")
    place, raw = _place(device, stream)
    with place:
        # one allocation: q_start, lengths, free head, then the token arrays
        flat = torch.empty(2 * requests + 2 + 2 * tokens, dtype=torch.int32, device=device)
        q_start, lens, head, slots, positions = flat.split_with_sizes((requests + 1, requests, 1, tokens, tokens))
        base = flat.data_ptr()
        B.bconv_block_tables(raw, requests, block_size, block_table.data_ptr(), width, stride,
                             context_lens.data_ptr(), new_lens.data_ptr(), free_blocks.data_ptr(), free_count,
                             free_head.data_ptr(), base + 4 * (2 * requests + 1), tokens,
                             base + 4 * (2 * requests + 2), base + 4 * (2 * requests + 2 + tokens), base,
                             base + 4 * (requests + 1))
    return BlockTables(slots, positions, q_start, lens, head)
