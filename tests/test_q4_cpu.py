"""Host-side checks of the 4-bit operators (no GPU): every function that
include/bconv_q4.h declares is exported and bound, descriptors and arguments
are refused with the documented codes before anything is launched, layouts are
as documented, and the references hold the formats' invariants."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import popcount_convolution_amd as pca
import q4_reference as ref
from popcount_convolution_amd import _binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, WORKSPACE = pca.BCONV_ERR_INVALID_ARGUMENT, pca.BCONV_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_binding.LIB_PATH):
        from popcount_convolution_amd import _build
        _build.build()
    return pca.load_library()


def test_header_symbols_exported(lib):
    text = open(os.path.join(ROOT, "include", "bconv_q4.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(bconv_[a-z0-9_]+)\s*\(", text)))
    assert len(names) == 9, names
    raw = ctypes.CDLL(_binding.LIB_PATH)
    assert not [n for n in names if not hasattr(raw, n)]
    assert not [n for n in names if not getattr(lib, n).argtypes]


def kv(**kw):
    d = dict(num_blocks=10, block_size=32, kv_heads=2, head_dim=128, group=64)
    d.update(kw)
    return pca.bconv_kv4_desc_t(*[d[n] for n, _ in pca.bconv_kv4_desc_t._fields_])


@pytest.mark.parametrize("bad", [
    dict(num_blocks=0), dict(num_blocks=1 << 27), dict(block_size=8), dict(block_size=24), dict(block_size=2048),
    dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=0), dict(head_dim=12), dict(head_dim=264),
    dict(group=16), dict(group=0), dict(group=256)])
def test_layout_refuses(lib, bad):
    with pytest.raises(pca.BconvError) as e:
        pca.bconv_kv4_layout(kv(**bad))
    assert e.value.status == INVALID


@pytest.mark.parametrize("dim,group,padded,groups", [
    (8, 32, 64, 2), (64, 128, 64, 1), (80, 32, 128, 4), (128, 64, 128, 2), (136, 128, 256, 2), (256, 32, 256, 8)])
def test_layout(lib, dim, group, padded, groups):
    L = pca.bconv_kv4_layout(kv(head_dim=dim, group=group))
    assert (L.dim_padded, L.groups, L.row_bytes) == (padded, groups, padded // 2)
    assert L.v_codes_offset == 32 * L.row_bytes and L.k_scales_offset == 64 * L.row_bytes
    assert L.v_scales_offset - L.k_scales_offset == 32 * groups * 4
    assert L.record_bytes == L.v_scales_offset + 32 * groups * 4
    assert L.pool_bytes == L.record_bytes * 2 * 10


def test_linear_create_refuses(lib):
    w, s = np.zeros((4, 4), np.uint32), np.ones((4, 1), np.float16)
    for args in ((0, 4, 32), (32, 0, 32), (32, 4, 48), ((1 << 20) + 1, 4, 32), (1 << 20, 1 << 20, 128)):
        with pytest.raises(pca.BconvError) as e:
            pca.bconv_q4_linear_create(*args, w, s)
        assert e.value.status == INVALID
    with pytest.raises(pca.BconvError) as e:
        pca.bconv_q4_linear_create(32, 4, 32, w, s, np.full((4, 1), 16, np.uint8))
    assert e.value.status == INVALID and "zeros[0]" in str(e.value)
    h = ctypes.c_void_p()
    d = _binding.bconv_q4_linear_desc_t(32, 4, 32)
    assert lib.bconv_q4_linear_create(d, None, s.ctypes.data, None, None, ctypes.byref(h)) == INVALID
    assert lib.bconv_q4_linear_create(None, None, None, None, None, ctypes.byref(h)) == INVALID
    assert lib.bconv_q4_linear_create(d, None, None, None, None, None) == INVALID
    assert lib.bconv_q4_linear_forward(None, None, 1, 0, None, 1, None, 1, None, 0) == INVALID
    assert lib.bconv_q4_linear_workspace_size(None, 1, 0, None) == INVALID
    assert lib.bconv_q4_linear_destroy(None) == pca.BCONV_OK


def test_append_refuses(lib):
    def call(d=None, pool=0x1000, tokens=1, dtype=0, k=0x2000, ks=(256, 128), v=0x3000, vs=(256, 128), slots=0x4000,
             ko=None, vo=None):
        with pytest.raises(pca.BconvError) as e:
            pca.bconv_kv4_append(d or kv(), None, pool, tokens, dtype, k, ks, v, vs, slots, ko, vo)
        assert e.value.status == INVALID
    call(d=kv(group=7))
    call(tokens=-1)
    call(dtype=3)
    call(pool=None)
    call(k=None)
    call(v=None)
    call(slots=None)
    call(pool=0x1001)
    call(k=0x2001)
    call(ko=0x2002)
    call(ks=(-1, 1))
    call(vs=(1, 1 << 41))
    call(tokens=1 << 30, d=kv(kv_heads=1024))
    pca.bconv_kv4_append(kv(), None, None, 0, 0, None, (0, 0), None, (0, 0), None)  # nothing to do


def attn(**kw):
    d = dict(pool=0x1000, q=0x2000, q_token_stride=512, q_head_stride=128, out=0x3000, lse=None, block_table=0x4000,
             context_lens=0x5000, q_start=None, requests=2, q_tokens=2, max_q=1, heads=4, table_width=8,
             table_stride=8, max_context=0, window=0, dtype=2, scale=0.1)
    d.update(kw)
    return pca.bconv_kv4_attention_t(*[d[n] for n, _ in pca.bconv_kv4_attention_t._fields_])


@pytest.mark.parametrize("bad", [
    dict(heads=3), dict(heads=0), dict(requests=-1), dict(q_tokens=-1), dict(q_tokens=3), dict(max_q=0),
    dict(q_tokens=4, max_q=1), dict(table_width=-1), dict(table_stride=7), dict(max_context=-1),
    dict(max_context=(1 << 30) + 1), dict(window=-1), dict(dtype=5), dict(q_token_stride=-1),
    dict(pool=None), dict(q=None), dict(out=None), dict(context_lens=None), dict(block_table=None),
    dict(pool=0x1004), dict(q=0x2001), dict(out=0x3001)])
def test_attention_refuses(lib, bad):
    with pytest.raises(pca.BconvError) as e:
        pca.bconv_kv4_attention(kv(), None, attn(**bad), 0x10000, 1 << 40)
    assert e.value.status == INVALID


def test_attention_workspace(lib):
    """Short contexts need none; a long axis with few rows is split, and a
    missing or short workspace is refused."""
    assert pca.bconv_kv4_attention_workspace_size(kv(), attn()) == 0
    long = attn(table_width=4096, table_stride=4096)
    need = pca.bconv_kv4_attention_workspace_size(kv(num_blocks=9000), long)
    assert need > 0
    for ws, size in ((None, 0), (0x10000, need - 1)):
        with pytest.raises(pca.BconvError) as e:
            pca.bconv_kv4_attention(kv(num_blocks=9000), None, long, ws, size)
        assert e.value.status == WORKSPACE
    assert pca.bconv_kv4_attention_workspace_size(kv(num_blocks=9000), attn(
        table_width=4096, table_stride=4096, max_context=100)) == 0
    pca.bconv_kv4_attention(kv(), None, attn(requests=0, q_tokens=0, q=None))
    with pytest.raises(pca.BconvError):
        pca.bconv_kv4_attention_workspace_size(kv(), None)


def test_block_tables_refuses(lib):
    def call(requests=2, block=16, table=0x1000, width=4, stride=4, ctx=0x2000, new=0x3000, free=0x4000, count=3,
             head=0x5000, out=0x6000, tokens=2, lens=None):
        with pytest.raises(pca.BconvError) as e:
            pca.bconv_block_tables(None, requests, block, table, width, stride, ctx, new, free, count, head, out,
                                   tokens, None, None, None, lens)
        assert e.value.status == INVALID
    call(requests=-1)
    call(requests=8193)
    call(block=17)
    call(block=8)
    call(table=None)
    call(width=-1)
    call(stride=3)
    call(ctx=None)
    call(new=None)
    call(free=None)
    call(count=-1)
    call(tokens=-1)
    call(head=None)
    call(out=None)
    call(out=0x5000)
    call(lens=0x2004)


# ------------------------------------------------------- the torch wrapper

def test_wrapper_refuses_host_and_mismatched_tensors():
    layer = object.__new__(pca.Q4Linear)
    layer.handle, layer.in_features, layer.out_features, layer.group = None, 16, 8, 32
    for x, match in ((torch.zeros(2, 15), "shape"), (torch.zeros(2, 16, dtype=torch.float64), "dtype"),
                     (torch.zeros(2, 16), "CUDA"), ([0.0] * 16, "torch tensor"),
                     (torch.zeros(16, 2).t(), "strides"), (torch.zeros(1, 16).expand(4, 16), "strides")):
        with pytest.raises(ValueError, match=match):
            layer.forward(x)
    with pytest.raises(ValueError, match="group"):
        pca.Q4Linear(in_features=8, out_features=2, weight_words=None, scales=None, group=16)
    with pytest.raises(ValueError, match="weight_words"):
        pca.Q4Linear(in_features=8, out_features=2, weight_words=np.zeros((2, 2), np.uint32), scales=None)
    with pytest.raises(ValueError, match="float16"):
        pca.Q4Linear(in_features=8, out_features=2, weight_words=np.zeros((2, 1), np.uint32),
                     scales=np.zeros((2, 1), np.float32))
    cache = object.__new__(pca.KV4Cache)
    cache.kv_heads, cache.head_dim, cache.device = 2, 64, torch.device("cuda:0")
    k, slots = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    for bad, match in (((k[:, :1], k, slots), "shape"), ((k, k[:2], slots), "tokens"),
                       ((k.double(), k.double(), slots), "dtype"), ((k, k.half(), slots), "dtype"),
                       ((k, k, slots), "CUDA"), ((k.transpose(0, 2).contiguous().transpose(0, 2), k, slots),
                                                 "contiguous")):
        with pytest.raises(ValueError, match=match):
            cache.append(*bad)
    q, table = torch.zeros(2, 4, 64), torch.zeros((2, 3), dtype=torch.int32)
    for bad, match in ((torch.zeros(2, 3, 64), "multiple"), (torch.zeros(2, 4, 32), "shape"), (q.double(), "dtype"),
                       (q, "CUDA"), (torch.zeros(2, 64), "shape")):
        with pytest.raises(ValueError, match=match):
            cache.attention(bad, table, slots[:2])
    with pytest.raises(ValueError, match="block_table"):
        pca.build_block_tables(torch.zeros(2, 3), slots, slots, slots, slots, block_size=16, tokens=1)
    with pytest.raises(ValueError, match="CUDA"):
        pca.build_block_tables(table, slots, slots, slots, slots, block_size=16, tokens=1)


def test_pack_codes():
    rng = np.random.default_rng(0)
    for k in (1, 7, 8, 9, 33):
        c = rng.integers(0, 16, (3, k))
        w = pca.pack_codes(c)
        assert w.dtype == np.uint32 and w.shape == (3, -(-k // 8))
        assert np.array_equal(ref.unpack_words(w, k), c)
    with pytest.raises(ValueError):
        pca.pack_codes(np.full((1, 1), 16))
    with pytest.raises(ValueError):
        pca.pack_codes(np.zeros(4))


# ---------------------------------------------------- the references' sense

def test_reference_quantise_invariants():
    """Every value comes back within half a step and the roundings of s and b,
    the extremes take codes near 0 and 15, a constant group comes back in fp16."""
    rng = np.random.default_rng(1)
    x = rng.normal(0, 2, (50, 3, 80)).astype(np.float32)
    c, s, b, val = ref.quantise(x, 32)
    step = np.repeat(s.astype(np.float64), 32, -1)[..., :80]
    mid = np.abs(np.repeat(b.astype(np.float64), 32, -1)[..., :80])
    assert (np.abs(val - x) <= step * (0.5 + 16 * 2.0 ** -11) + mid * 2.0 ** -10).all()
    assert c.max() == 15 and c.min() == 0
    c, s, b, val = ref.quantise(np.full((1, 64), 0.3, np.float32), 64)
    assert (c == 8).all() and not s.any() and (val == np.float32(np.float16(0.3))).all()


def test_reference_attention_invariants():
    """Equal keys average the values; one visible token returns its value."""
    kx, vx = np.ones((32, 1, 8)), np.random.default_rng(2).normal(0, 1, (32, 1, 8))
    table = np.array([[1, 0]], np.int32)
    q = np.ones((1, 1, 8))
    out, lse, _ = ref.attention(q, kx, vx, np.ones((32, 1)), table, [20], [1], block_size=16, kv_heads=1, scale=0.5)
    seen = np.concatenate([vx[16:, 0], vx[:4, 0]])
    assert np.allclose(out[0, 0], seen.mean(0)) and np.allclose(lse, 4 + np.log(20))
    out, *_ = ref.attention(q, kx, vx, np.ones((32, 1)), table, [20], [1], block_size=16, kv_heads=1, scale=0.5,
                            window=1)
    assert np.allclose(out[0, 0], vx[3, 0])


def test_numbers_past_32_bits():
    """Numbers that an int32 does not hold are refused, not wrapped."""
    with pytest.raises(ValueError, match="num_blocks"):
        pca.KV4Cache(2 ** 32 + 1, 16, 1, 64)
    with pytest.raises(ValueError, match="block_size"):
        pca.KV4Cache(1, 2 ** 32 + 16, 1, 64)
