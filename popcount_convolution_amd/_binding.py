"""ctypes binding of libbconv.so.

Functions carry the names of the C ABI in ``include/bconv.h`` and only
marshal arguments: device pointers are plain integers (or torch tensors, whose
``data_ptr()`` is taken), host arrays are numpy arrays.  Nothing here
computes any step of the forward pass; if the shared library is missing every
entry point raises ``BconvLibraryMissing``.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbconv.so")

# bconv_status_t
BCONV_OK = 0
BCONV_ERR_INVALID_ARGUMENT = 1
BCONV_ERR_UNSUPPORTED = 2
BCONV_ERR_WORKSPACE = 3
BCONV_ERR_ALLOC = 4
BCONV_ERR_HIP = 5
# bconv_type_t
BCONV_BINARY_WEIGHTS = 0
BCONV_XNOR = 1
BCONV_AND = 2
# flags
BCONV_FLAG_NONE = 0
BCONV_FLAG_USE_BETA_SCALING = 1
BCONV_FLAG_INT8_MFMA = 2
BCONV_FLAG_BETA_VALID_TAPS = 4
BCONV_FLAG_FP4_MFMA = 8
# bconv_neuron_t
BCONV_NEURON_NONE = 0
BCONV_NEURON_RELU = 1
NEURON_NAMES = ("none", "relu", "leaky_relu", "linear", "sigmoid", "hard_sigmoid", "tanh", "absolute", "softplus",
                "softsign", "elu", "clamp")

TYPE_CODES = {"binary_weights": BCONV_BINARY_WEIGHTS, "xnor": BCONV_XNOR, "and": BCONV_AND}
NEURON_CODES = {name: code for code, name in enumerate(NEURON_NAMES)}
SIZE_MAX = ctypes.c_size_t(-1).value
BCONV_SCRATCH_MAX_BYTES = 16 << 20


class BconvLibraryMissing(RuntimeError):
    pass


class BconvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_name(status)}: {message}")
        self.status = status


class bconv_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "in_h", "in_w", "in_c", "out_c", "kernel_h", "kernel_w", "stride_h", "stride_w",
        "pad_h", "pad_w", "groups", "neuron")] + [("scale_value", ctypes.c_float)] + \
        [("pad_h_end", ctypes.c_int32), ("pad_w_end", ctypes.c_int32),
         ("neuron_a", ctypes.c_float), ("neuron_b", ctypes.c_float)]


class bconv_workspace_layout_t(ctypes.Structure):
    _fields_ = [("bits_offset", ctypes.c_size_t), ("bits_rows", ctypes.c_int32),
                ("bits_cols", ctypes.c_int32), ("bits_words", ctypes.c_int32),
                ("bits_pad_h", ctypes.c_int32), ("bits_pad_w", ctypes.c_int32),
                ("a_map_offset", ctypes.c_size_t), ("beta_offset", ctypes.c_size_t),
                ("total_bytes", ctypes.c_size_t)]


# bconv_dtype_t
BCONV_F32 = 0
BCONV_F16 = 1
BCONV_BF16 = 2


class bconv_q4_linear_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("in_features", "out_features", "group")]


class bconv_kv4_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_blocks", "block_size", "kv_heads", "head_dim", "group")]


class bconv_kv4_layout_t(ctypes.Structure):
    _fields_ = [("pool_bytes", ctypes.c_size_t), ("record_bytes", ctypes.c_size_t), ("row_bytes", ctypes.c_int32),
                ("dim_padded", ctypes.c_int32), ("groups", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("v_codes_offset", ctypes.c_size_t), ("k_scales_offset", ctypes.c_size_t),
                ("v_scales_offset", ctypes.c_size_t)]


class bconv_kv4_attention_t(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("context_lens", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("requests", ctypes.c_int32), ("q_tokens", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("table_width", ctypes.c_int32), ("table_stride", ctypes.c_int32),
                ("max_context", ctypes.c_int32), ("window", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class bconv_mx4_linear_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("experts", "in_features", "out_features")]


class bconv_mx4_rows_t(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("x_rows", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("choices", ctypes.c_int32), ("offsets", ctypes.c_void_p),
                ("order", ctypes.c_void_p)]


_lib = None


def load_library(path: Optional[str] = None):
    """Load libbconv.so and declare its signatures (raises if it is missing)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise BconvLibraryMissing(
            f"{p} is not built: run __graft_entry__.build() (hipcc --offload-arch=gfx950)")
    lib = ctypes.CDLL(p)
    vp, i32, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
    i64 = ctypes.c_int64
    st = ctypes.c_int
    fp = ctypes.POINTER(ctypes.c_float)
    up = ctypes.POINTER(ctypes.c_uint32)
    sigs = {
        "bconv_validate_desc": (st, [ctypes.POINTER(bconv_desc_t), i32, u32]),
        "bconv_create": (st, [ctypes.POINTER(bconv_desc_t), up, fp, fp, fp, fp, i32, u32,
                              ctypes.POINTER(vp)]),
        "bconv_create_fc": (st, [i32, i32, i32, i32, i32, ctypes.c_float, up, fp, fp, fp, fp,
                                 i32, u32, ctypes.POINTER(vp)]),
        "bconv_get_info": (st, [vp] + [ctypes.POINTER(i32)] * 4),
        "bconv_workspace_size": (st, [vp, i32, ctypes.POINTER(sz)]),
        "bconv_workspace_layout": (st, [vp, i32, ctypes.POINTER(bconv_workspace_layout_t)]),
        "bconv_forward": (st, [vp, vp, i32, vp, vp, vp, sz]),
        "bconv_forward_noalloc": (st, [vp, vp, i32, vp, vp]),
        "bconv_forward_accum": (st, [vp, vp, i32, vp, vp, vp, sz]),
        "bconv_forward_profiled": (st, [vp, vp, i32, vp, vp, vp, sz, vp, vp, vp, vp]),
        "bconv_forward_bits": (st, [vp, vp, i32, vp, vp, vp, sz]),
        "bconv_forward_bits_profiled": (st, [vp, vp, i32, vp, vp, vp, sz, vp, vp, vp, vp]),
        "bconv_main_kernel": (ctypes.c_char_p, [vp, i32]),
        "bconv_forward_packed": (st, [vp, vp, i32, vp, vp, vp, sz]),
        "bconv_forward_packed_bits": (st, [vp, vp, i32, vp, vp, vp, sz]),
        "bconv_calibrate_popcount": (st, [vp, i32, i32, u32, vp]),
        "bconv_destroy": (st, [vp]),
        "bconv_status_string": (ctypes.c_char_p, [st]),
        "bconv_last_error": (ctypes.c_char_p, []),
        "bconv_q4_linear_create": (st, [ctypes.POINTER(bconv_q4_linear_desc_t), up, vp, vp, fp, ctypes.POINTER(vp)]),
        "bconv_q4_linear_workspace_size": (st, [vp, i32, i32, ctypes.POINTER(sz)]),
        "bconv_q4_linear_forward": (st, [vp, vp, i32, i32, vp, i64, vp, i64, vp, sz]),
        "bconv_q4_linear_destroy": (st, [vp]),
        "bconv_kv4_layout": (st, [ctypes.POINTER(bconv_kv4_desc_t), ctypes.POINTER(bconv_kv4_layout_t)]),
        "bconv_kv4_append": (st, [ctypes.POINTER(bconv_kv4_desc_t), vp, vp, i32, i32, vp, i64, i64, vp, i64, i64, vp,
                                  vp, vp]),
        "bconv_kv4_attention_workspace_size": (st, [ctypes.POINTER(bconv_kv4_desc_t),
                                                    ctypes.POINTER(bconv_kv4_attention_t), ctypes.POINTER(sz)]),
        "bconv_kv4_attention": (st, [ctypes.POINTER(bconv_kv4_desc_t), vp, ctypes.POINTER(bconv_kv4_attention_t), vp,
                                     sz]),
        "bconv_block_tables": (st, [vp, i32, i32, vp, i32, i32, vp, vp, vp, i32, vp, vp, i32, vp, vp, vp, vp]),
        "bconv_mx4_quantize": (st, [vp, i32, i32, i32, vp, i64, vp, vp, vp]),
        "bconv_mx4_linear_create": (st, [ctypes.POINTER(bconv_mx4_linear_desc_t), vp, vp, vp, vp, ctypes.POINTER(vp)]),
        "bconv_mx4_linear_workspace_size": (st, [vp, ctypes.POINTER(bconv_mx4_rows_t), ctypes.POINTER(sz)]),
        "bconv_mx4_linear_forward": (st, [vp, vp, ctypes.POINTER(bconv_mx4_rows_t), vp, sz]),
        "bconv_mx4_linear_destroy": (st, [vp]),
        "bconv_expert_sort_workspace_size": (st, [i32, i32, ctypes.POINTER(sz)]),
        "bconv_expert_sort": (st, [vp, i32, i32, i32, vp, vp, vp, vp, vp, sz]),
        "bconv_expert_gather": (st, [vp, i32, i32, i32, i32, vp, i64, vp, vp, vp]),
        "bconv_expert_combine": (st, [vp, i32, i32, i32, i32, vp, i64, vp, i32, vp, vp]),
        "bconv_expert_combine_backward": (st, [vp, i32, i32, i32, i32, vp, i64, vp, i64, vp, vp, i32, vp, vp, vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def status_name(s: int) -> str:
    try:
        return load_library().bconv_status_string(s).decode()
    except BconvLibraryMissing:
        return f"status {s}"


def _check(status: int) -> None:
    if status != BCONV_OK:
        raise BconvError(status, bconv_last_error())


def _host_f32(a) -> Optional[ctypes.POINTER(ctypes.c_float)]:
    if a is None:
        return None
    arr = np.ascontiguousarray(a, dtype=np.float32)
    return arr, arr.ctypes.data_as(ctypes.POINTER(ctypes.c_float))


def _ptr(x) -> Optional[int]:
    """Device pointer of a torch tensor or a plain integer address."""
    if x is None or type(x) is int:
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


def make_desc(in_h, in_w, in_c, out_c, kernel_h, kernel_w, stride_h=1, stride_w=1, pad_h=0,
              pad_w=0, groups=1, neuron=BCONV_NEURON_NONE, scale_value=1.0, pad_h_end=None,
              pad_w_end=None, neuron_a=0.0, neuron_b=0.0) -> bconv_desc_t:
    """Trailing padding defaults to the leading one (symmetric padding)."""
    return bconv_desc_t(in_h, in_w, in_c, out_c, kernel_h, kernel_w, stride_h, stride_w, pad_h,
                        pad_w, groups, neuron, scale_value, pad_h if pad_h_end is None else pad_h_end,
                        pad_w if pad_w_end is None else pad_w_end, neuron_a, neuron_b)


def bconv_validate_desc(desc: bconv_desc_t, type: int, flags: int) -> int:
    return load_library().bconv_validate_desc(ctypes.byref(desc), type, flags)


def bconv_create(desc: bconv_desc_t, weight_bits: np.ndarray, output_scale=None, output_bias=None,
                 input_scale=None, input_bias=None, type: int = BCONV_XNOR,
                 flags: int = BCONV_FLAG_NONE) -> int:
    lib = load_library()
    wb = np.ascontiguousarray(weight_bits, dtype=np.uint32)
    keep = [_host_f32(a) for a in (output_scale, output_bias, input_scale, input_bias)]
    ptrs = [k[1] if k else None for k in keep]
    h = ctypes.c_void_p()
    _check(lib.bconv_create(ctypes.byref(desc), wb.ctypes.data_as(ctypes.POINTER(ctypes.c_uint32)),
                            *ptrs, type, flags, ctypes.byref(h)))
    return h.value


def bconv_create_fc(in_h, in_w, in_c, out_c, neuron, scale_value, weight_bits, output_scale=None,
                    output_bias=None, input_scale=None, input_bias=None, type=BCONV_XNOR,
                    flags=BCONV_FLAG_NONE) -> int:
    lib = load_library()
    wb = np.ascontiguousarray(weight_bits, dtype=np.uint32)
    keep = [_host_f32(a) for a in (output_scale, output_bias, input_scale, input_bias)]
    ptrs = [k[1] if k else None for k in keep]
    h = ctypes.c_void_p()
    _check(lib.bconv_create_fc(in_h, in_w, in_c, out_c, neuron, scale_value,
                               wb.ctypes.data_as(ctypes.POINTER(ctypes.c_uint32)), *ptrs, type,
                               flags, ctypes.byref(h)))
    return h.value


def bconv_get_info(h: int):
    vals = [ctypes.c_int32() for _ in range(4)]
    _check(load_library().bconv_get_info(h, *[ctypes.byref(v) for v in vals]))
    return tuple(v.value for v in vals)


def bconv_workspace_size(h: int, n: int) -> int:
    b = ctypes.c_size_t()
    _check(load_library().bconv_workspace_size(h, n, ctypes.byref(b)))
    return b.value


def bconv_workspace_layout(h: int, n: int) -> dict:
    L = bconv_workspace_layout_t()
    _check(load_library().bconv_workspace_layout(h, n, ctypes.byref(L)))
    d = {name: getattr(L, name) for name, _ in L._fields_}
    for k in ("bits_offset", "a_map_offset", "beta_offset"):
        if d[k] == SIZE_MAX:
            d[k] = None
    return d


def bconv_forward(h: int, stream, n: int, inp, out, workspace, workspace_bytes: int) -> None:
    _check(load_library().bconv_forward(h, _ptr(stream), n, _ptr(inp), _ptr(out), _ptr(workspace),
                                        workspace_bytes))


def bconv_forward_noalloc(h: int, stream, n: int, inp, out) -> None:
    _check(load_library().bconv_forward_noalloc(h, _ptr(stream), n, _ptr(inp), _ptr(out)))


def bconv_forward_accum(h: int, stream, n: int, inp, acc, workspace, workspace_bytes: int) -> None:
    _check(load_library().bconv_forward_accum(h, _ptr(stream), n, _ptr(inp), _ptr(acc),
                                              _ptr(workspace), workspace_bytes))


def bconv_forward_profiled(h: int, stream, n: int, inp, out, workspace, workspace_bytes: int,
                           main_begin=None, main_end=None, input_begin=None, input_end=None) -> None:
    _check(load_library().bconv_forward_profiled(h, _ptr(stream), n, _ptr(inp), _ptr(out),
                                                 _ptr(workspace), workspace_bytes,
                                                 _ptr(main_begin), _ptr(main_end),
                                                 _ptr(input_begin), _ptr(input_end)))


def bconv_forward_bits(h: int, stream, n: int, inp, out_bits, workspace, workspace_bytes: int) -> None:
    _check(load_library().bconv_forward_bits(h, _ptr(stream), n, _ptr(inp), _ptr(out_bits), _ptr(workspace),
                                             workspace_bytes))


def bconv_forward_bits_profiled(h: int, stream, n: int, inp, out_bits, workspace, workspace_bytes: int,
                                main_begin=None, main_end=None, input_begin=None, input_end=None) -> None:
    _check(load_library().bconv_forward_bits_profiled(h, _ptr(stream), n, _ptr(inp), _ptr(out_bits),
                                                      _ptr(workspace), workspace_bytes,
                                                      _ptr(main_begin), _ptr(main_end),
                                                      _ptr(input_begin), _ptr(input_end)))


def bconv_forward_packed(h: int, stream, n: int, in_bits, out, workspace, workspace_bytes: int) -> None:
    _check(load_library().bconv_forward_packed(h, _ptr(stream), n, _ptr(in_bits), _ptr(out), _ptr(workspace),
                                               workspace_bytes))


def bconv_forward_packed_bits(h: int, stream, n: int, in_bits, out_bits, workspace, workspace_bytes: int) -> None:
    _check(load_library().bconv_forward_packed_bits(h, _ptr(stream), n, _ptr(in_bits), _ptr(out_bits),
                                                    _ptr(workspace), workspace_bytes))


def bconv_main_kernel(h: int, n: int) -> str:
    return load_library().bconv_main_kernel(h, n).decode()


def bconv_calibrate_popcount(stream, blocks: int, iters: int, seed: int, sink) -> None:
    _check(load_library().bconv_calibrate_popcount(_ptr(stream), blocks, iters, seed, _ptr(sink)))


def bconv_destroy(h: int) -> None:
    _check(load_library().bconv_destroy(h))


def bconv_status_string(s: int) -> str:
    return load_library().bconv_status_string(s).decode()


def bconv_last_error() -> str:
    return load_library().bconv_last_error().decode()


def bconv_q4_linear_create(in_features: int, out_features: int, group: int, weight_words, scales, zeros=None,
                           bias=None) -> int:
    """Host arrays: uint32 words, fp16 scales, uint8 zeros or None, float32 bias or None."""
    desc = bconv_q4_linear_desc_t(in_features, out_features, group)
    ww = np.ascontiguousarray(weight_words, dtype=np.uint32)
    sc = np.ascontiguousarray(scales, dtype=np.float16)
    zs = None if zeros is None else np.ascontiguousarray(zeros, dtype=np.uint8)
    b = _host_f32(bias)
    h = ctypes.c_void_p()
    _check(load_library().bconv_q4_linear_create(
        ctypes.byref(desc), ww.ctypes.data_as(ctypes.POINTER(ctypes.c_uint32)), sc.ctypes.data,
        None if zs is None else zs.ctypes.data, b[1] if b else None, ctypes.byref(h)))
    return h.value


def bconv_q4_linear_workspace_size(h: int, rows: int, dtype: int) -> int:
    b = ctypes.c_size_t()
    _check(load_library().bconv_q4_linear_workspace_size(h, rows, dtype, ctypes.byref(b)))
    return b.value


def bconv_q4_linear_forward(h: int, stream, rows: int, dtype: int, x, ldx: int, y, ldy: int, workspace=None,
                            workspace_bytes: int = 0) -> None:
    st = (_lib or load_library()).bconv_q4_linear_forward(h, stream, rows, dtype, _ptr(x), ldx, _ptr(y), ldy,
                                                          _ptr(workspace), workspace_bytes)
    if st:
        _check(st)


def bconv_q4_linear_destroy(h: int) -> None:
    _check(load_library().bconv_q4_linear_destroy(h))


def bconv_kv4_layout(desc: bconv_kv4_desc_t) -> bconv_kv4_layout_t:
    layout = bconv_kv4_layout_t()
    _check(load_library().bconv_kv4_layout(ctypes.byref(desc), ctypes.byref(layout)))
    return layout


def bconv_kv4_append(desc: bconv_kv4_desc_t, stream, pool, tokens: int, dtype: int, k, k_strides, v, v_strides, slots,
                     k_out=None, v_out=None) -> None:
    st = (_lib or load_library()).bconv_kv4_append(desc, stream, _ptr(pool), tokens, dtype, _ptr(k), *k_strides,
                                                   _ptr(v), *v_strides, _ptr(slots), _ptr(k_out), _ptr(v_out))
    if st:
        _check(st)


def bconv_kv4_attention_workspace_size(desc: bconv_kv4_desc_t, args: bconv_kv4_attention_t) -> int:
    b = ctypes.c_size_t()
    _check(load_library().bconv_kv4_attention_workspace_size(desc, args, ctypes.byref(b)))
    return b.value


def bconv_kv4_attention(desc: bconv_kv4_desc_t, stream, args: bconv_kv4_attention_t, workspace=None,
                        workspace_bytes: int = 0) -> None:
    st = (_lib or load_library()).bconv_kv4_attention(desc, stream, args, _ptr(workspace), workspace_bytes)
    if st:
        _check(st)


def bconv_block_tables(stream, requests: int, block_size: int, block_table, table_width: int, table_stride: int,
                       context_lens, new_lens, free_blocks, free_count: int, free_head, free_head_out, tokens: int,
                       slots=None, positions=None, q_start=None, context_lens_out=None) -> None:
    st = (_lib or load_library()).bconv_block_tables(
        stream, requests, block_size, _ptr(block_table), table_width, table_stride, _ptr(context_lens),
        _ptr(new_lens), _ptr(free_blocks), free_count, _ptr(free_head), _ptr(free_head_out), tokens, _ptr(slots),
        _ptr(positions), _ptr(q_start), _ptr(context_lens_out))
    if st:
        _check(st)


def bconv_mx4_quantize(stream, rows: int, cols: int, dtype: int, x, ldx: int, codes, scales, values=None) -> None:
    st = (_lib or load_library()).bconv_mx4_quantize(stream, rows, cols, dtype, _ptr(x), ldx, _ptr(codes),
                                                     _ptr(scales), _ptr(values))
    if st:
        _check(st)


def bconv_mx4_linear_create(experts: int, in_features: int, out_features: int, stream, codes, scales, bias=None) -> int:
    """Device arrays: uint8 codes and scales, float32 bias or None."""
    desc = bconv_mx4_linear_desc_t(experts, in_features, out_features)
    h = ctypes.c_void_p()
    _check(load_library().bconv_mx4_linear_create(ctypes.byref(desc), _ptr(stream), _ptr(codes), _ptr(scales),
                                                  _ptr(bias), ctypes.byref(h)))
    return h.value


def bconv_mx4_linear_workspace_size(h: int, args: bconv_mx4_rows_t) -> int:
    b = ctypes.c_size_t()
    _check(load_library().bconv_mx4_linear_workspace_size(h, args, ctypes.byref(b)))
    return b.value


def bconv_mx4_linear_forward(h: int, stream, args: bconv_mx4_rows_t, workspace=None, workspace_bytes: int = 0) -> None:
    st = (_lib or load_library()).bconv_mx4_linear_forward(h, stream, args, _ptr(workspace), workspace_bytes)
    if st:
        _check(st)


def bconv_mx4_linear_destroy(h: int) -> None:
    _check(load_library().bconv_mx4_linear_destroy(h))


def bconv_expert_sort_workspace_size(pairs: int, experts: int) -> int:
    b = ctypes.c_size_t()
    _check(load_library().bconv_expert_sort_workspace_size(pairs, experts, ctypes.byref(b)))
    return b.value


def bconv_expert_sort(stream, pairs: int, experts: int, id_bytes: int, ids, offsets, order, position, workspace=None,
                      workspace_bytes: int = 0) -> None:
    st = (_lib or load_library()).bconv_expert_sort(stream, pairs, experts, id_bytes, _ptr(ids), _ptr(offsets),
                                                    _ptr(order), _ptr(position), _ptr(workspace), workspace_bytes)
    if st:
        _check(st)


def bconv_expert_gather(stream, tokens: int, choices: int, width: int, dtype: int, x, ldx: int, order, position,
                        rows) -> None:
    st = (_lib or load_library()).bconv_expert_gather(stream, tokens, choices, width, dtype, _ptr(x), ldx, _ptr(order),
                                                      _ptr(position), _ptr(rows))
    if st:
        _check(st)


def bconv_expert_combine(stream, tokens: int, choices: int, width: int, dtype: int, rows, ldr: int, position,
                         weight_dtype: int, weights, y) -> None:
    st = (_lib or load_library()).bconv_expert_combine(stream, tokens, choices, width, dtype, _ptr(rows), ldr,
                                                       _ptr(position), weight_dtype, _ptr(weights), _ptr(y))
    if st:
        _check(st)


def bconv_expert_combine_backward(stream, tokens: int, choices: int, width: int, dtype: int, dy, ldd: int, rows,
                                  ldr: int, order, position, weight_dtype: int, weights, d_rows,
                                  d_weights=None) -> None:
    st = (_lib or load_library()).bconv_expert_combine_backward(
        stream, tokens, choices, width, dtype, _ptr(dy), ldd, _ptr(rows), ldr, _ptr(order), _ptr(position),
        weight_dtype, _ptr(weights), _ptr(d_rows), _ptr(d_weights))
    if st:
        _check(st)
