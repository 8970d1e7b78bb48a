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

_DTYPES: dict = {}


def _dtype_codes() -> dict:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: B.BCONV_F32, torch.float16: B.BCONV_F16, torch.bfloat16: B.BCONV_BF16})
    return _DTYPES


def _dtype_code(t, name: str) -> int:
    code = _dtype_codes().get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: dtype {t.dtype} is not one of torch.float32, torch.float16, torch.bfloat16")
    return code


def _need_tensor(t, name: str) -> None:
    import torch
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a torch tensor is required, got {type(t).__name__}")


def _need_cuda(t, name: str, device=None) -> None:
    if t.device.type != "cuda":
        raise ValueError(f"{name}: a CUDA (HIP) device tensor is required, got device {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, not on {device}")


def _need_int32(t, name: str, shape, device) -> None:
    """A contiguous int32 device tensor of exactly ``shape``."""
    import torch
    _need_tensor(t, name)
    if t.dtype != torch.int32:
        raise ValueError(f"{name}: dtype {t.dtype} is not torch.int32")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: the tensor must be contiguous")
    _need_cuda(t, name, device)


def _need_dense(t, name: str, shape, dtype, device) -> None:
    _need_tensor(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} is not {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: the tensor must be contiguous")
    _need_cuda(t, name, device)


def _need_rows(t, name: str, heads: int, dim: int) -> int:
    """[tokens, heads, dim] with contiguous channels; token and head strides
    are free.  Returns the tokens."""
    _need_tensor(t, name)
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not (tokens, {heads}, {dim})")
    if dim > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: channels must be contiguous (stride {t.stride(2)})")
    return t.shape[0]


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
    import torch
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


_STAY = contextlib.nullcontext()


def _place(device, stream):
    """(context to allocate and launch in, raw stream): nothing to enter when
    the call goes to the current device's current stream."""
    import torch
    if stream is None:
        s = torch.cuda.current_stream(device)
        if device.index == torch.cuda.current_device():
            return _STAY, s.cuda_stream
    else:
        if stream.device != device:
            raise ValueError(f"stream: on {stream.device}, the tensors are on {device}")
        s = stream
    return _on(device, s), s.cuda_stream


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
    float32, float16 or bfloat16 rows and sums in float32.
    """

    def __init__(self, *, in_features: int, out_features: int, weight_words, scales, zeros=None, bias=None,
                 group: int = 128):
        self.handle = None
        if group not in (32, 64, 128):
            raise ValueError(f"group: {group} is not 32, 64 or 128")
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
        self.handle = B.bconv_q4_linear_create(in_features, out_features, group, weight_words, scales, zeros, bias)

    def workspace_bytes(self, rows: int, dtype) -> int:
        return B.bconv_q4_linear_workspace_size(self.handle, rows, _dtype_codes()[dtype])

    def forward(self, x, out=None, workspace=None, stream=None):
        """``[..., in_features]`` -> ``[..., out_features]`` of the same type.
        A 2-d x or out may have any row stride; others must be contiguous."""
        import torch
        _need_tensor(x, "input")
        if x.dim() < 1 or x.shape[-1] != self.in_features:
            raise ValueError(f"input: shape {tuple(x.shape)} does not end in {self.in_features}")
        code = _dtype_code(x, "input")
        rows, ldx = _row_stride(x, "input")
        device = x.device
        _need_cuda(x, "input")
        place, raw = _place(device, stream)
        with place:
            if out is None:
                out = torch.empty(x.shape[:-1] + (self.out_features,), dtype=x.dtype, device=device)
                ldy = self.out_features
            else:
                _need_tensor(out, "output")
                if tuple(out.shape) != tuple(x.shape[:-1]) + (self.out_features,):
                    raise ValueError(f"output: shape {tuple(out.shape)} != "
                                     f"{tuple(x.shape[:-1]) + (self.out_features,)}")
                if out.dtype != x.dtype:
                    raise ValueError(f"output: dtype {out.dtype} is not {x.dtype}")
                _need_cuda(out, "output", device)
                ldy = _row_stride(out, "output")[1]
            if rows == 0:
                return out
            need = B.bconv_q4_linear_workspace_size(self.handle, rows, code)
            if workspace is None:
                if need:
                    workspace = torch.empty(need, dtype=torch.uint8, device=device)
            else:
                _need_workspace(workspace, need, device)
            B.bconv_q4_linear_forward(self.handle, raw, rows, code, x, ldx, out, ldy, workspace, need)
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
        import torch
        self.desc = B.bconv_kv4_desc_t(num_blocks, block_size, kv_heads, head_dim, group)
        self.layout = B.bconv_kv4_layout(self.desc)
        self.num_blocks, self.block_size, self.kv_heads = num_blocks, block_size, kv_heads
        self.head_dim, self.group = head_dim, group
        self.pool = torch.zeros(self.layout.pool_bytes, dtype=torch.uint8, device=device or "cuda")
        _need_cuda(self.pool, "device")
        self.device = self.pool.device

    def append(self, k, v, slots, *, values: bool = False, k_out=None, v_out=None, stream=None):
        """Writes new rows ``[tokens, kv_heads, head_dim]`` at ``slots`` (int32
        ``[tokens]``, block * block_size + offset; slots outside the pool are
        skipped).  With ``values`` (or ``k_out`` / ``v_out``) returns the pair of
        dense tensors that the cache now stands for."""
        import torch
        tokens = _need_rows(k, "k", self.kv_heads, self.head_dim)
        if _need_rows(v, "v", self.kv_heads, self.head_dim) != tokens:
            raise ValueError(f"v: {v.shape[0]} tokens, k has {tokens}")
        code = _dtype_code(k, "k")
        if v.dtype != k.dtype:
            raise ValueError(f"v: dtype {v.dtype} is not {k.dtype}")
        _need_cuda(k, "k", self.device)
        _need_cuda(v, "v", self.device)
        _need_int32(slots, "slots", (tokens,), self.device)
        place, raw = _place(self.device, stream)
        with place:
            shape = (tokens, self.kv_heads, self.head_dim)
            if k_out is not None:
                _need_dense(k_out, "k_out", shape, k.dtype, self.device)
            elif values:
                k_out = torch.empty(shape, dtype=k.dtype, device=self.device)
            if v_out is not None:
                _need_dense(v_out, "v_out", shape, k.dtype, self.device)
            elif values:
                v_out = torch.empty(shape, dtype=k.dtype, device=self.device)
            if tokens:
                B.bconv_kv4_append(self.desc, raw, self.pool, tokens, code, k, k.stride()[:2], v, v.stride()[:2],
                                   slots, k_out, v_out)
        return (k_out, v_out) if k_out is not None or v_out is not None else None

    def attention(self, q, block_table, context_lens, *, q_start=None, max_q: Optional[int] = None,
                  max_context: int = 0, scale: Optional[float] = None, window: int = 0, out=None, lse=None,
                  workspace=None, stream=None):
        """``softmax(scale q K^T + mask) V`` for ``q`` ``[tokens, heads, head_dim]``.

        ``block_table``: int32 ``[requests, width]``; ``context_lens``: int32
        ``[requests]``, cached tokens with the new ones; ``q_start``: int32
        ``[requests + 1]`` prefix sums of the requests' queries, with ``max_q`` the
        most of one request, or None for the same number each.  ``max_context``
        bounds the context lengths (the table's width by default).  ``scale``
        defaults to ``head_dim ** -0.5``; ``window`` > 0 limits a query to that many
        last positions.  ``lse``: float32 ``[tokens, heads]`` to fill."""
        import torch
        _need_tensor(q, "q")
        if q.dim() != 3 or q.shape[1] % self.kv_heads or not q.shape[1]:
            raise ValueError(f"q: shape {tuple(q.shape)} is not (tokens, a multiple of {self.kv_heads}, "
                             f"{self.head_dim})")
        tokens, heads = q.shape[0], q.shape[1]
        _need_rows(q, "q", heads, self.head_dim)
        code = _dtype_code(q, "q")
        device = self.device
        _need_cuda(q, "q", device)
        _need_tensor(block_table, "block_table")
        if block_table.dtype != torch.int32 or block_table.dim() != 2:
            raise ValueError(f"block_table: {block_table.dtype} of shape {tuple(block_table.shape)} is not int32 "
                             "(requests, width)")
        _need_cuda(block_table, "block_table", device)
        requests, width = block_table.shape
        if width > 1 and block_table.stride(1) != 1 or requests > 1 and block_table.stride(0) < width:
            raise ValueError("block_table: rows must be contiguous and must not overlap")
        _need_int32(context_lens, "context_lens", (requests,), device)
        if q_start is not None:
            _need_int32(q_start, "q_start", (requests + 1,), device)
            if max_q is None:
                max_q = max(1, tokens)
        else:
            if requests and tokens % requests:
                raise ValueError(f"q: {tokens} tokens are not a multiple of {requests} requests (pass q_start)")
            if max_q is None:
                max_q = max(1, tokens // requests if requests else 1)
        place, raw = _place(device, stream)
        with place:
            if out is None:
                out = torch.empty((tokens, heads, self.head_dim), dtype=q.dtype, device=device)
            else:
                _need_dense(out, "out", (tokens, heads, self.head_dim), q.dtype, device)
            if lse is not None:
                _need_dense(lse, "lse", (tokens, heads), torch.float32, device)
            if not tokens or not requests:
                return out
            stride = block_table.stride(0) if requests > 1 else max(width, 1)
            args = B.bconv_kv4_attention_t(
                self.pool.data_ptr(), q.data_ptr(), q.stride(0), q.stride(1), out.data_ptr(),
                None if lse is None else lse.data_ptr(), block_table.data_ptr(), context_lens.data_ptr(),
                None if q_start is None else q_start.data_ptr(), requests, tokens, max_q, heads, width, stride,
                max_context, window, code, self.head_dim ** -0.5 if scale is None else scale)
            need = B.bconv_kv4_attention_workspace_size(self.desc, args)
            if workspace is None:
                if need:
                    workspace = torch.empty(need, dtype=torch.uint8, device=device)
            else:
                _need_workspace(workspace, need, device)
            B.bconv_kv4_attention(self.desc, raw, args, workspace, need)
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
    import torch
    _need_tensor(block_table, "block_table")
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise ValueError(f"block_table: {block_table.dtype} of shape {tuple(block_table.shape)} is not int32 "
                         "(requests, width)")
    _need_cuda(block_table, "block_table")
    requests, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1 or requests > 1 and block_table.stride(0) < width:
        raise ValueError("block_table: rows must be contiguous and must not overlap")
    device = block_table.device
    _need_int32(context_lens, "context_lens", (requests,), device)
    _need_int32(new_lens, "new_lens", (requests,), device)
    _need_tensor(free_blocks, "free_blocks")
    _need_int32(free_blocks, "free_blocks", (free_blocks.numel(),), device)
    _need_int32(free_head, "free_head", (1,), device)
    if tokens < 0:
        raise ValueError(f"tokens: {tokens} is negative")
    place, raw = _place(device, stream)
    with place:
        # one allocation: q_start, lengths, free head, then the token arrays
        flat = torch.empty(2 * requests + 2 + 2 * tokens, dtype=torch.int32, device=device)
        q_start, lens, head, slots, positions = flat.split((requests + 1, requests, 1, tokens, tokens))
        stride = block_table.stride(0) if requests > 1 else max(width, 1)
        base = flat.data_ptr()
        B.bconv_block_tables(raw, requests, block_size, block_table, width, stride, context_lens, new_lens,
                             free_blocks, free_blocks.numel(), free_head, base + 4 * (2 * requests + 1), tokens,
                             base + 4 * (2 * requests + 2), base + 4 * (2 * requests + 2 + tokens), base,
                             base + 4 * (requests + 1))
    return BlockTables(slots, positions, q_start, lens, head)
