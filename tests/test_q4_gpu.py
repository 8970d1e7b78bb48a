"""4-bit linear layers, cache, attention and block tables on the GPU against
plain 64-bit references (q4_reference.py), at the sizes, strides and masks
where they can go wrong."""

import numpy as np
import pytest
import torch

import popcount_convolution_amd as pca
import q4_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pca.load_library()
    return torch.device("cuda:0")


def say(*a):
    print(*a, flush=True)


def host(t):
    return t.to(torch.float64).cpu().numpy()


# ------------------------------------------------------------------ linear

def make_linear(rng, k, n, group, zeros, bias):
    codes = rng.integers(0, 16, (n, k))
    groups = -(-k // group)
    scales = (rng.uniform(0.3, 1.5, (n, groups)) * 0.02).astype(np.float16)
    zs = rng.integers(0, 16, (n, groups)).astype(np.uint8) if zeros else None
    b = rng.normal(0, 1, n).astype(np.float32) if bias else None
    words = pca.pack_codes(codes)
    # nibbles past in_features are ignored
    if k % 8:
        words[:, -1] |= np.uint32((0xffffffff << (4 * (k % 8))) & 0xffffffff)
    layer = pca.Q4Linear(in_features=k, out_features=n, weight_words=words, scales=scales, zeros=zs, bias=b,
                         group=group)
    return layer, words, scales, zs, b


def check_linear(layer, w, x, y, group, dtype):
    words, scales, zs, b = w
    k = layer.in_features
    xh = host(x).reshape(-1, k)
    want, mass = ref.linear(xh, words, scales, zs, b, group)
    bound = ref.linear_bound(want, mass, b, k, group, dtype)
    err = np.abs(host(y).reshape(-1, layer.out_features) - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(err / bound)} of its bound"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k,n,group,zeros,bias", [
    (1, 1, 1, 32, False, False),
    (1, 8, 5, 128, True, True),
    (1, 32, 16, 32, False, False),
    (1, 512, 512, 32, False, True),
    (1, 4096, 96, 128, False, False),
    (1, 5000, 67, 64, True, False),
    (2, 129, 31, 64, True, False),
    (3, 127, 33, 128, False, True),
    (5, 1000, 130, 32, True, True),
    (15, 100, 17, 32, False, False),
    (16, 256, 64, 64, False, True),
    (17, 300, 48, 128, True, True),
    (32, 640, 80, 32, True, False),
    (33, 1025, 65, 64, False, False),
    (48, 384, 200, 128, False, True),
    (64, 2048, 128, 128, True, False),
    (65, 1111, 129, 64, True, True),
    (130, 777, 257, 32, False, True),
    (200, 1536, 300, 128, False, False),
    (257, 520, 140, 64, True, True),
    (520, 260, 530, 128, True, False),
])
def test_linear(dev, dtype, rows, k, n, group, zeros, bias):
    say("linear", dtype, rows, k, n, group, zeros, bias)
    rng = np.random.default_rng(rows * 1000003 + k * 1009 + n)
    layer, *w = make_linear(rng, k, n, group, zeros, bias)
    x = torch.from_numpy(rng.normal(0, 1, (rows, k)).astype(np.float32)).to(dev).to(DT[dtype])
    y = layer.forward(x)
    torch.cuda.synchronize()
    assert y.dtype == x.dtype and y.shape == (rows, n)
    check_linear(layer, w, x, y, group, dtype)
    layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k,n,group,zeros,bias", [
    (17, 8200, 4100, 64, True, True),
    (33, 5000, 4400, 32, False, False),
    (50, 4100, 4111, 128, True, False),
    (65, 3333, 4000, 128, False, True),
    (130, 2049, 3500, 64, False, False),
    (130, 2049, 3500, 32, True, True),
    (300, 1100, 3100, 128, True, False),
    (300, 1100, 3100, 64, True, True),
    (2000, 300, 1400, 32, False, True),   # inputs too short to split
    (2000, 300, 1400, 128, True, False),
])
def test_linear_many_rows(dev, dtype, rows, k, n, group, zeros, bias):
    """Products large enough for the many-row kernel: each width of its column
    blocks, split and whole inputs, ragged last tiles and chunks."""
    say("linear many", dtype, rows, k, n, group, zeros, bias)
    rng = np.random.default_rng(rows * 1000003 + k * 1009 + n)
    layer, *w = make_linear(rng, k, n, group, zeros, bias)
    assert layer.workspace_bytes(rows, DT[dtype]) > 0  # it takes that kernel
    x = torch.from_numpy(rng.normal(0, 1, (rows, k)).astype(np.float32)).to(dev).to(DT[dtype])
    buf = torch.full((rows, n + 3), 7.0, device=dev, dtype=DT[dtype])
    ws = torch.full((layer.workspace_bytes(rows, DT[dtype]),), 0xff, dtype=torch.uint8, device=dev)
    y = layer.forward(x, out=buf[:, :n], workspace=ws)
    torch.cuda.synchronize()
    check_linear(layer, w, x, y, group, dtype)
    assert bool((buf[:, n:] == 7.0).all())
    # strided, misaligned rows give the same
    wide = torch.zeros((rows, k + 3), device=dev, dtype=DT[dtype])
    wide[:, 1:k + 1] = x
    assert torch.equal(layer.forward(wide[:, 1:k + 1]), y)
    layer.close()


@pytest.mark.parametrize("dtype", ["f16", "f32", "bf16"])
def test_linear_many_rows_nonfinite(dev, dtype):
    """A bad row leaves the others alone in the many-row kernel too."""
    rng = np.random.default_rng(15)
    layer, *_ = make_linear(rng, 1100, 3100, 64, True, False)
    x = rng.normal(0, 1, (300, 1100)).astype(np.float32)
    clean = x.copy()
    x[100, 7], x[101, 1099] = np.inf, np.nan
    y = host(layer.forward(torch.from_numpy(x).to(dev).to(DT[dtype])))
    z = host(layer.forward(torch.from_numpy(clean).to(dev).to(DT[dtype])))
    assert not np.isfinite(y[100]).any() and np.isnan(y[101]).all()
    assert np.array_equal(np.delete(y, [100, 101], 0), np.delete(z, [100, 101], 0))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [1, 7, 40, 150])
@pytest.mark.parametrize("ldx,offset,ldy", [(211, 0, 77), (208, 0, 80), (217, 3, 90), (224, 1, 71)])
def test_linear_strides(dev, dtype, rows, ldx, offset, ldy):
    """Rows at any element alignment and stride; what lies between the output
    rows stays as it was."""
    say("linear strides", dtype, rows, ldx, offset, ldy)
    rng = np.random.default_rng(rows + ldx)
    k, n = 200, 70
    layer, *w = make_linear(rng, k, n, 64, True, True)
    buf = torch.from_numpy(rng.normal(0, 1, rows * ldx + offset + 8).astype(np.float32)).to(dev).to(DT[dtype])
    x = buf[offset:offset + rows * ldx].view(rows, ldx)[:, :k]
    ybuf = torch.full((rows * ldy + offset,), 7.0, device=dev, dtype=DT[dtype])
    y = ybuf[offset:].view(rows, ldy)[:, :n]
    got = layer.forward(x, out=y)
    torch.cuda.synchronize()
    assert got is y
    check_linear(layer, w, x, y, 64, dtype)
    assert bool((ybuf[offset:].view(rows, ldy)[:, n:] == 7.0).all()) and bool((ybuf[:offset] == 7.0).all())


def test_linear_same_sign(dev):
    """Inputs of one sign (as after a ReLU): the offset of the codes is then at
    its largest against the result."""
    rng = np.random.default_rng(5)
    for dtype in DT:
        for rows in (1, 20, 100):
            say("same sign", dtype, rows)
            layer, *w = make_linear(rng, 2000, 64 if rows < 100 else 5000, 128, True, False)
            x = torch.from_numpy(np.abs(rng.normal(0, 1, (rows, 2000))).astype(np.float32)).to(dev).to(DT[dtype])
            check_linear(layer, w, x, layer.forward(x), 128, dtype)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("rows", [2, 70])
def test_linear_nonfinite(dev, dtype, rows):
    """fp16 and fp32 rows follow IEEE arithmetic; a bad row leaves the others."""
    rng = np.random.default_rng(11)
    layer, words, scales, _, _ = make_linear(rng, 256, 40, 64, False, False)
    x = rng.normal(0, 1, (rows, 256)).astype(np.float32)
    x[1, 3], clean = np.inf, x.copy()
    clean[1, 3] = 0
    y = host(layer.forward(torch.from_numpy(x).to(dev).to(DT[dtype])))
    c = ref.unpack_words(words, 256)[:, 3].astype(int) - 8
    want = np.where(c > 0, np.inf, np.where(c < 0, -np.inf, np.nan))
    assert np.array_equal(y[1], want, equal_nan=True)
    z = host(layer.forward(torch.from_numpy(clean).to(dev).to(DT[dtype])))
    assert np.array_equal(np.delete(y, 1, 0), np.delete(z, 1, 0))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,n", [(1, 80), (13, 5000), (70, 300), (70, 9000)])
def test_linear_fp32_range(dev, rows, n, zeros):
    """fp32 rows from 1e-30 to 1e30 with values of one row 2^20 apart: a value is
    split to 2^-24 of itself or 2^-39 of its row's largest, whichever is more."""
    say("fp32 range", rows, n, zeros)
    rng = np.random.default_rng(rows + n)
    layer, *w = make_linear(rng, 2000, n, 64, zeros, False)
    x = rng.normal(0, 1, (rows, 2000)) * 2.0 ** rng.integers(-20, 1, (rows, 2000))
    x = (x * 10.0 ** np.linspace(-30, 30, rows)[:, None]).astype(np.float32)
    y = layer.forward(torch.from_numpy(x).to(dev))
    xh = x.astype(np.float64)
    want, mass = ref.linear(xh, *w, 64)
    weights = ref.linear(np.ones((1, 2000)), *w, 64)[1]
    bound = (ref.linear_bound(want, mass, None, 2000, 64, "f32") + 2.0 ** -24 * mass +
             2.0 ** -39 * np.abs(xh).max(1, keepdims=True) * weights)
    bad = ~(np.abs(host(y) - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off"


@pytest.mark.parametrize("rows", [2, 70])
def test_linear_nonfinite_bf16(dev, rows):
    """A bf16 row with an infinity gives NaN in that row alone."""
    rng = np.random.default_rng(12)
    layer, *_ = make_linear(rng, 256, 40, 64, True, False)
    x = rng.normal(0, 1, (rows, 256)).astype(np.float32)
    x[1, 200] = -np.inf
    y = host(layer.forward(torch.from_numpy(x).to(dev).bfloat16()))
    assert np.isnan(y[1]).all() and np.isfinite(np.delete(y, 1, 0)).all()


def test_linear_rows_agree(dev):
    """A row's result does not depend on its place in a batch of the same size."""
    rng = np.random.default_rng(13)
    layer, *_ = make_linear(rng, 1000, 100, 64, False, True)
    for rows in (40, 300, 3000):
        x = torch.from_numpy(rng.normal(0, 1, (rows, 1000)).astype(np.float32)).to(dev).bfloat16()
        perm = torch.randperm(rows, device=dev)
        assert torch.equal(layer.forward(x)[perm], layer.forward(x[perm].contiguous()))
        assert torch.equal(layer.forward(x), layer.forward(x))


def test_linear_shapes_and_streams(dev):
    rng = np.random.default_rng(14)
    layer, *w = make_linear(rng, 96, 40, 32, False, False)
    x = torch.randn(3, 5, 96, device=dev).half()
    assert layer.forward(x).shape == (3, 5, 40)
    assert layer.forward(x[:0]).shape == (0, 5, 40)
    assert layer.forward(x[0, 0]).shape == (40,)
    s = torch.cuda.Stream()
    big = torch.randn(4096, 96, device=dev)
    s.wait_stream(torch.cuda.current_stream())
    y = layer.forward(big, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, layer.forward(big))
    assert layer.workspace_bytes(150, torch.bfloat16) == 0  # few rows for so small a layer: no workspace


def test_linear_columns_of_one_buffer(dev):
    """x and y as columns of one buffer share no element; columns that do are
    refused."""
    rng = np.random.default_rng(16)
    layer, *w = make_linear(rng, 64, 48, 32, False, False)
    buf = torch.randn(5, 200, device=dev)
    x = buf[:, :64].clone()
    for left, right in ((buf[:, :64], buf[:, 64:112]), (buf[:, 60:124], buf[:, 5:53])):
        left.copy_(x)
        assert torch.equal(layer.forward(left, out=right), layer.forward(x))
    for left, right in ((buf[:, :64], buf[:, 63:111]), (buf[:, 40:104], buf[:, 0:48])):
        with pytest.raises(pca.BconvError):
            layer.forward(left, out=right)


def test_linear_rows_past_32_bits(dev):
    """Row offsets beyond 2^32 bytes and 2^31 elements."""
    rng = np.random.default_rng(17)
    layer, *w = make_linear(rng, 300, 40, 64, True, False)
    buf = torch.empty((3, (1 << 30) + 64), dtype=torch.bfloat16, device=dev)
    x = buf[:, :300]
    x.copy_(torch.randn(3, 300, device=dev))
    check_linear(layer, w, x, layer.forward(x), 64, "bf16")


# ------------------------------------------------------------------- cache

def rows_of(rng, tokens, heads, dim, kind):
    x = rng.normal(0, 1, (tokens, heads, dim))
    if kind == "outliers":
        x[..., rng.random(dim) < 0.1] *= 30
    elif kind == "constant":
        x[...] = 0.1234
    elif kind == "tiny":
        x *= 1e-6
    elif kind == "huge":
        x *= 3e4
    elif kind == "special" and tokens:
        flat = x.reshape(-1)
        flat[rng.integers(0, flat.size, max(1, flat.size // 9))] = np.inf
        flat[rng.integers(0, flat.size, max(1, flat.size // 9))] = -np.inf
        flat[rng.integers(0, flat.size, max(1, flat.size // 9))] = np.nan
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,heads,dim,group,block,kind", [
    (1, 1, 8, 32, 16, "normal"),
    (1, 2, 64, 32, 16, "outliers"),
    (3, 3, 64, 64, 32, "constant"),
    (5, 1, 64, 128, 16, "tiny"),
    (33, 8, 128, 64, 32, "outliers"),
    (17, 2, 128, 32, 16, "special"),
    (40, 1, 128, 128, 64, "huge"),
    (21, 5, 80, 32, 16, "outliers"),
    (19, 2, 96, 64, 16, "normal"),
    (9, 3, 104, 128, 16, "special"),
    (12, 2, 256, 32, 16, "outliers"),
    (50, 1, 200, 64, 128, "normal"),
    (7, 4, 256, 128, 16, "constant"),
])
def test_append(dev, dtype, tokens, heads, dim, group, block, kind):
    """Codes, steps and midpoints in the pool equal the format's own steps bit
    for bit; skipped tokens leave the pool as it was; strided views."""
    say("append", dtype, tokens, heads, dim, group, block, kind)
    rng = np.random.default_rng(tokens * 7919 + dim)
    blocks = -(-tokens // block) + 2
    cache = pca.KV4Cache(blocks, block, heads, dim, group=group)
    k = torch.from_numpy(rows_of(rng, tokens, 3 * heads, dim, kind)).to(dev).to(DT[dtype])
    v = torch.from_numpy(rows_of(rng, tokens, 3 * heads, dim, "normal")).to(dev).to(DT[dtype])
    k, v = k[:, heads:2 * heads], v[:, ::3]
    slots = rng.permutation(blocks * block)[:tokens].astype(np.int32)
    skip = rng.random(tokens) < 0.2
    bad = rng.choice([-1, -7, blocks * block, 2 ** 31 - 1], tokens)
    given = np.where(skip, bad, slots).astype(np.int32)
    vk, vv = cache.append(k, v, torch.from_numpy(given).to(dev), values=True)
    torch.cuda.synchronize()
    got = ref.read_pool(cache.pool.cpu().numpy(), cache.layout, blocks, block, heads, dim)
    groups = -(-dim // group)
    for side, x, val in ((got[0], k, vk), (got[1], v, vv)):
        c, s, b, want = ref.quantise(x.float().cpu().numpy(), group)
        at = slots[~skip]
        assert np.array_equal(side["codes"][at], c[~skip])
        assert np.array_equal(side["s"][at][..., :groups].view(np.uint16), s[~skip].view(np.uint16))
        assert np.array_equal(side["b"][at][..., :groups].view(np.uint16), b[~skip].view(np.uint16))
        assert torch.equal(val.cpu(), torch.from_numpy(want).to(DT[dtype]))
        rest = np.setdiff1d(np.arange(blocks * block), at)
        assert not side["s"][rest].any() and not side["codes"][rest].any()


def test_append_without_values_and_empty(dev):
    cache = pca.KV4Cache(4, 16, 2, 64)
    k = torch.randn(5, 2, 64, device=dev)
    slots = torch.arange(5, dtype=torch.int32, device=dev)
    assert cache.append(k, k, slots) is None
    other = pca.KV4Cache(4, 16, 2, 64)
    out = torch.empty(5, 2, 64, device=dev)
    assert other.append(k, k, slots, k_out=out)[0] is out
    assert torch.equal(cache.pool, other.pool)
    cache.append(k[:0], k[:0], slots[:0])
    # an odd element offset: no 16-byte loads
    flat = torch.empty(5 * 2 * 64 + 1, device=dev)
    flat[1:] = k.flatten()
    third = pca.KV4Cache(4, 16, 2, 64)
    third.append(flat[1:].view(5, 2, 64), k, slots)
    assert torch.equal(cache.pool, third.pool)


# --------------------------------------------------------------- attention

def make_cache(rng, dev, lens, heads, dim, group, block, spare=2):
    """A filled cache, its shuffled table, and its values in 64 bits."""
    per = [-(-int(n) // block) for n in lens]
    blocks = sum(per) + spare
    order = rng.permutation(blocks)
    width = max(per + [1]) + 1
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for r, n in enumerate(per):
        table[r, :n] = order[at:at + n]
        at += n
    cache = pca.KV4Cache(blocks, block, heads, dim, group=group)
    # rows that no request owns hold garbage, infinities and NaN among it
    cache.pool.copy_(torch.from_numpy(rng.integers(0, 256, cache.pool.numel(), dtype=np.uint8)))
    slots = np.concatenate([table[r, np.arange(n) // block].astype(np.int64) * block + np.arange(n) % block
                            for r, n in enumerate(lens)] + [np.zeros(0, np.int64)])
    k = rng.normal(0, 1, (slots.size, heads, dim)).astype(np.float32)
    k[..., rng.random(dim) < 0.05] *= 5
    v = rng.normal(0.3, 1, (slots.size, heads, dim)).astype(np.float32)
    cache.append(torch.from_numpy(k).to(dev), torch.from_numpy(v).to(dev),
                 torch.from_numpy(slots.astype(np.int32)).to(dev))
    kx = np.full((blocks * block, heads, dim), np.nan)
    vx, vs = kx.copy(), np.full((blocks * block, heads), np.nan)
    kx[slots] = ref.quantise(k, group)[3]
    _, s, _, val = ref.quantise(v, group)
    vx[slots], vs[slots] = val, s.astype(np.float64).max(-1) if slots.size else 0
    return cache, table, kx, vx, vs


def check_attention(rng, dev, dtype, lens, counts, heads, kv_heads, dim, group, block, window=0, uniform=False,
                    q=None, table=None, made=None, max_context=0, **kw):
    cache, tab, kx, vx, vs = made or make_cache(rng, dev, lens, kv_heads, dim, group, block)
    table = tab if table is None else table
    total = int(sum(counts))
    if q is None:
        q = torch.from_numpy(rng.normal(0, 1.2, (total, heads, dim)).astype(np.float32)).to(dev).to(DT[dtype])
    starts = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(dev)
    lse = torch.full((total, heads), 99.0, device=dev)
    t = torch.from_numpy(table).to(dev)
    n = torch.from_numpy(np.asarray(lens, np.int32)).to(dev)
    out = cache.attention(q, t, n, q_start=None if uniform else starts, max_q=None if uniform else max(counts),
                          window=window, lse=lse, max_context=max_context, **kw)
    torch.cuda.synchronize()
    want, wlse, terms = ref.attention(host(q), kx, vx, vs, table, lens, counts, block_size=block, kv_heads=kv_heads,
                                      scale=kw.get("scale", dim ** -0.5), window=window, num_blocks=cache.num_blocks)
    bound = ref.attention_bound(want, terms, dim, int(max(list(lens) + [1])), dtype)
    err = np.abs(host(out) - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(err / np.maximum(bound, 1e-300))}"
    got = host(lse)
    empty = np.isneginf(wlse)
    assert np.array_equal(empty, np.isneginf(got))
    assert not host(out)[empty].any()
    parts = 3 if dtype == "f32" else 1
    lse_bound = ref.EPS * (dim * parts + 16) * 8 * terms[0] + 2.0 ** -19 * (1 + np.abs(np.where(empty, 0, wlse)))
    assert (np.abs(got[~empty] - wlse[~empty]) <= lse_bound[~empty]).all()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens,heads,kv_heads,dim,group,block", [
    ([1], 1, 1, 64, 64, 16),
    ([7, 0, 31, 32, 33], 2, 1, 64, 32, 16),
    ([100], 8, 2, 128, 64, 32),
    ([513, 1, 260], 4, 4, 128, 32, 16),
    ([1500, 40], 16, 1, 128, 128, 64),
    ([90, 200], 20, 1, 64, 128, 16),
    ([300, 17], 14, 2, 80, 32, 16),
    ([65, 129], 6, 3, 96, 64, 128),
    ([250], 5, 5, 8, 32, 16),
    ([333, 64], 8, 2, 256, 64, 32),
    ([100, 50], 8, 4, 200, 32, 16),
    ([140], 4, 2, 256, 128, 256),
    ([2300, 700], 40, 1, 104, 128, 1024),
    ([20000, 3, 9000], 16, 1, 64, 64, 64),     # dozens of parts
])
def test_attention_decode(dev, dtype, lens, heads, kv_heads, dim, group, block):
    """One query a request: lengths of zero, one and odd ones, pages that end
    inside a tile, several parts, more heads a group than a tile holds."""
    say("decode", dtype, lens, heads, kv_heads, dim, group, block)
    rng = np.random.default_rng(sum(lens) * 31 + heads * 7 + dim)
    check_attention(rng, dev, dtype, lens, [1] * len(lens), heads, kv_heads, dim, group, block, uniform=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens,counts,heads,kv_heads,dim,group,block,window", [
    ([40, 9, 70], [3, 9, 0], 2, 1, 64, 32, 16, 0),
    ([200, 33], [50, 33], 4, 2, 128, 64, 32, 0),
    ([129, 5, 64], [17, 1, 20], 6, 2, 128, 128, 16, 13),
    ([700, 300], [40, 130], 3, 3, 80, 32, 16, 100),
    ([150], [70], 7, 1, 256, 64, 64, 1),
    ([620, 90], [5, 90], 8, 1, 64, 64, 16, 33),
    ([2, 5], [4, 5], 2, 2, 64, 64, 16, 0),   # more queries than cached tokens: the first see nothing
    ([1200, 1100], [2, 1], 16, 2, 128, 32, 64, 600),
])
def test_attention_ragged(dev, dtype, lens, counts, heads, kv_heads, dim, group, block, window):
    say("ragged", dtype, lens, counts, heads, kv_heads, dim, group, block, window)
    rng = np.random.default_rng(sum(lens) * 13 + sum(counts))
    check_attention(rng, dev, dtype, lens, counts, heads, kv_heads, dim, group, block, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_large_logits(dev, dtype):
    """Logits that rise along the context, so that the running maximum moves,
    and ones far below it; a negative scale."""
    rng = np.random.default_rng(3)
    for scale in (0.5, 2.0, -0.5):
        check_attention(rng, dev, dtype, [400, 33], [1, 1], 8, 2, 64, 32, 16, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 64), (64, 32), (128, 128), (120, 64), (128, 32), (256, 128), (200, 64), (256, 32)])
@pytest.mark.parametrize("heads,counts,window", [
    (1, [1, 1, 1], 0), (2, [2, 0, 1], 0), (1, [4, 3, 2], 0), (3, [1, 1, 1], 9), (4, [1, 1, 1], 0), (1, [4, 2, 4], 5),
    (1, [5, 1, 3], 0),
])
def test_attention_few_columns(dev, dtype, dim, group, heads, counts, window):
    """One to five (query, head) pairs a request and key/value head: up to four
    of them share their softmax between lanes."""
    say("few columns", dtype, dim, group, heads, counts, window)
    rng = np.random.default_rng(dim * 100 + group + heads * 10 + sum(counts))
    check_attention(rng, dev, dtype, [703, 2, 45], counts, 2 * heads, 2, dim, group, 16, window)


@pytest.mark.parametrize("heads", [2, 32])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (200, 64)])
def test_attention_fp32_steps(dev, dim, group, heads):
    """Values whose steps span 1e-3 to 1e3, growing and shrinking along the
    context, under queries of 1e-15 to 1e15 with the scale that undoes it."""
    rng = np.random.default_rng(dim + heads)
    for order in (1, -1):
        for size in (1e-15, 1.0, 1e15):
            n, block = 900, 16
            cache, table, kx, vx, vs = make_cache(rng, dev, [n], 2, dim, group, block)
            slots = (table[0, np.arange(n) // block].astype(np.int64) * block + np.arange(n) % block)
            k = rng.normal(0, 1, (n, 2, dim)).astype(np.float32)
            v = (rng.normal(0, 1, k.shape) * 10.0 ** np.linspace(-3, 3, n)[::order, None, None]).astype(np.float32)
            cache.append(torch.from_numpy(k).to(dev), torch.from_numpy(v).to(dev),
                         torch.from_numpy(slots.astype(np.int32)).to(dev))
            kx[slots] = ref.quantise(k, group)[3]
            _, s, _, val = ref.quantise(v, group)
            vx[slots], vs[slots] = val, s.astype(np.float64).max(-1)
            q = torch.from_numpy((rng.normal(0, 1, (1, heads, dim)) * size).astype(np.float32)).to(dev)
            check_attention(rng, dev, "f32", [n], [1], heads, 2, dim, group, block, uniform=True, q=q,
                            made=(cache, table, kx, vx, vs), scale=dim ** -0.5 / size)


@pytest.mark.parametrize("heads", [4, 32])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64), (128, 128), (256, 32)])
def test_attention_bf16_probabilities(dev, dim, group, heads):
    """A bf16 result's error is its own rounding's, to a quarter: probabilities
    have 11 bits, an eighth of bf16's error, on the sum of terms up to a few times
    the result.  One token's steps are 2^12 of the others', early or late."""
    rng = np.random.default_rng(dim + heads + group)
    n, block = 700, 32
    for at in (None, 3, 650):
        cache, table, kx, vx, vs = make_cache(rng, dev, [n], 2, dim, group, block)
        slots = (table[0, np.arange(n) // block].astype(np.int64) * block + np.arange(n) % block)
        k = rng.normal(0, 1, (n, 2, dim)).astype(np.float32)
        v = rng.normal(0, 1, k.shape).astype(np.float32)
        if at is not None:
            v[at] *= 2.0 ** 12
        cache.append(torch.from_numpy(k).to(dev), torch.from_numpy(v).to(dev),
                     torch.from_numpy(slots.astype(np.int32)).to(dev))
        kx[slots], vx[slots] = ref.quantise(k, group)[3], ref.quantise(v, group)[3]
        q = torch.from_numpy(rng.normal(0, 1.5, (1, heads, dim)).astype(np.float32)).to(dev).bfloat16()
        out = cache.attention(q, torch.from_numpy(table).to(dev), torch.tensor([n], dtype=torch.int32, device=dev))
        want = ref.attention(host(q), kx, vx, vs, table, [n], [1], block_size=block, kv_heads=2, scale=dim ** -0.5,
                             num_blocks=cache.num_blocks)[0]
        best = torch.from_numpy(want).bfloat16().double().numpy()
        rms = lambda e: np.sqrt((e ** 2).mean(-1)).mean()  # noqa: E731
        assert rms(host(out) - want) <= 1.25 * rms(best - want)


def test_attention_lowest_logits(dev):
    """Logits far below any mask's usual value are still those of a softmax: a
    lone token has probability one."""
    for heads in (1, 8):
        cache = pca.KV4Cache(2, 16, 1, 64, group=64)
        k, v = torch.ones(1, 1, 64, device=dev), torch.randn(1, 1, 64, device=dev)
        _, value = cache.append(k, v, torch.zeros(1, dtype=torch.int32, device=dev), values=True)
        q = torch.full((1, heads, 64), -1e35, device=dev)
        out = cache.attention(q, torch.zeros(1, 1, dtype=torch.int32, device=dev),
                              torch.ones(1, dtype=torch.int32, device=dev))
        assert float((out - value).abs().max()) <= 2.0 ** -20 * float(value.abs().max())


def test_attention_missing_blocks(dev):
    """Blocks outside the pool and positions past the table are masked; a
    request all of whose blocks are missing sees nothing."""
    rng = np.random.default_rng(4)
    for dtype in DT:
        lens = [100, 70, 90]
        made = make_cache(rng, dev, lens, 2, 64, 32, 16)
        table = made[1].copy()
        table[0, 2] = -1
        table[0, 5] = made[0].num_blocks
        table[1, :] = -5
        table[2, 3] = 2 ** 31 - 1
        check_attention(rng, dev, dtype, lens, [1, 1, 1], 4, 2, 64, 32, 16, table=table, made=made, uniform=True)
        check_attention(rng, dev, dtype, lens, [5, 3, 8], 4, 2, 64, 32, 16, table=np.ascontiguousarray(table[:, :4]),
                        made=made)


def test_attention_strided_queries(dev):
    rng = np.random.default_rng(6)
    for dtype in DT:
        lens = [77, 20]
        made = make_cache(rng, dev, lens, 2, 64, 32, 16)
        base = torch.randn(2, 9, 64 + 3, device=dev).to(DT[dtype])
        for q in (base[:, 1:5, 3:], base[:, ::2, :64][:, :4], base[:, 4:5, :64].expand(2, 4, 64)):
            check_attention(rng, dev, dtype, lens, [1, 1], 4, 2, 64, 32, 16, q=q, made=made, uniform=True)


def test_attention_bounds_and_offsets(dev):
    """max_context below the table's width splits the axis differently and gives
    the same result; queries that q_start leaves out stay as they were."""
    rng = np.random.default_rng(8)
    lens = [600, 100]
    made = make_cache(rng, dev, lens, 1, 128, 64, 16)
    cache, table = made[0], made[1]
    wide = np.full((2, 4000), -1, np.int32)
    wide[:, :table.shape[1]] = table
    a = check_attention(rng, dev, "f32", lens, [1, 1], 4, 1, 128, 64, 16, made=made, table=wide, uniform=True,
                        q=torch.ones(2, 4, 128, device=dev))
    b = check_attention(rng, dev, "f32", lens, [1, 1], 4, 1, 128, 64, 16, made=made, uniform=True, max_context=600,
                        q=torch.ones(2, 4, 128, device=dev))
    assert torch.allclose(a, b, rtol=1e-5, atol=1e-5)
    q = torch.randn(5, 4, 128, device=dev)
    out = torch.full((5, 4, 128), 3.0, device=dev)
    starts = torch.tensor([1, 3, 4], dtype=torch.int32, device=dev)
    cache.attention(q, torch.from_numpy(table).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                    q_start=starts, max_q=2, out=out)
    assert bool((out[0] == 3).all()) and bool((out[4] == 3).all()) and not bool((out[1:4] == 3).any())


def test_cache_past_32_bits(dev):
    """Blocks beyond 4 GiB of the pool: written and read where they are."""
    rng = np.random.default_rng(18)
    blocks = (5 << 30) // pca.bconv_kv4_layout(pca.bconv_kv4_desc_t(1, 64, 8, 128, 64)).record_bytes // 8
    high, low = pca.KV4Cache(blocks, 64, 8, 128), pca.KV4Cache(4, 64, 8, 128)
    k, v = torch.randn(150, 8, 128, device=dev), torch.randn(150, 8, 128, device=dev)
    pos = torch.arange(150, dtype=torch.int32, device=dev)
    ids = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=dev)
    far = ids + (blocks - 4)
    for cache, table in ((high, far), (low, ids)):
        cache.append(k, v, table[0][pos // 64] * 64 + pos % 64)
    q, lens = torch.randn(1, 32, 128, device=dev), torch.tensor([150], dtype=torch.int32, device=dev)
    assert torch.equal(high.attention(q, far, lens), low.attention(q, ids, lens))
    assert not high.pool[:1 << 30].any() and float(low.attention(q, ids, lens).abs().sum()) > 0


def test_attention_numbers_past_32_bits(dev):
    """Bounds that an int32 does not hold are refused, not wrapped."""
    cache, q = pca.KV4Cache(2, 16, 1, 64), torch.zeros(1, 1, 64, device=dev)
    table, lens = torch.zeros(1, 2, dtype=torch.int32, device=dev), torch.ones(1, dtype=torch.int32, device=dev)
    for name in ("max_context", "window", "max_q"):
        with pytest.raises(ValueError, match=name):
            cache.attention(q, table, lens, **{name: 2 ** 32 + 5})
    with pytest.raises(ValueError, match="block_size"):
        pca.build_block_tables(table, lens, lens, lens, lens, block_size=2 ** 32 + 16, tokens=1)


def test_attention_nan_query(dev):
    """A NaN query gives NaN for its own head alone."""
    rng = np.random.default_rng(9)
    cache, table, *_ = make_cache(rng, dev, [50], 2, 64, 64, 16)
    q = torch.randn(1, 4, 64, device=dev)
    clean = cache.attention(q, torch.from_numpy(table).to(dev), torch.tensor([50], dtype=torch.int32, device=dev))
    q[0, 1, 5] = float("nan")
    out = cache.attention(q, torch.from_numpy(table).to(dev), torch.tensor([50], dtype=torch.int32, device=dev))
    assert bool(out[0, 1].isnan().all())
    for h in (0, 2, 3):
        assert torch.equal(out[0, h], clean[0, h])


# ------------------------------------------------------------ block tables

@pytest.mark.parametrize("requests,ctx,new,block,free,extra", [
    (1, 0, 1, 16, 10, 0),
    (3, 40, 5, 16, 10, 4),
    (32, 500, 1, 32, 40, 0),
    (300, 200, 60, 16, 2000, 7),
    (300, 200, 60, 16, 100, 0),     # the free list runs out
    (1000, 50, 3, 64, 1000, 0),
    (8192, 30, 2, 16, 9000, 1),
    (2, 0, 5000, 16, 700, 0),
    (4, 100, 0, 16, 3, 5),
])
def test_block_tables(dev, requests, ctx, new, block, free, extra):
    say("tables", requests, ctx, new, block, free, extra)
    rng = np.random.default_rng(requests + new)
    c = rng.integers(0, ctx + 1, requests).astype(np.int32)
    n = rng.integers(0, new + 1, requests).astype(np.int32)
    if new:
        n[0] = new
    if requests > 2:
        c[1], n[2] = -3, -1  # negative lengths count as 0
    need = -(-(np.maximum(c, 0) + np.maximum(n, 0)) // block)
    width = max(1, int(need.max()) - (1 if requests == 3 else 0))  # too narrow once
    have = -(-np.maximum(c, 0) // block)
    table = np.full((requests, width + 2), -9, np.int32)
    for r in range(requests):
        table[r, :min(width, have[r])] = rng.integers(0, 5000, min(width, have[r]))
    if requests > 2:
        table[0, :1] = -1
    blocks = rng.permutation(free + 50)[:free].astype(np.int32)
    tokens = int(np.maximum(n, 0).sum()) + extra
    head = 1 if free > 1 else 0
    want = ref.block_tables(table[:, :width], c, n, blocks, head, block, tokens)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    t = up(table)
    got = pca.build_block_tables(t[:, :width], up(c), up(n), up(blocks), up(np.array([head], np.int32)),
                                 block_size=block, tokens=tokens)
    torch.cuda.synchronize()
    for name, value in (("table", t[:, :width]), ("slots", got.slots), ("positions", got.positions),
                        ("q_start", got.q_start), ("context_lens", got.context_lens), ("free_head", got.free_head)):
        assert np.array_equal(value.cpu().numpy(), want[name]), name
    assert bool((t[:, width:] == -9).all())


def test_block_tables_fewer_entries_and_empty(dev):
    """A slot map shorter than the new tokens still gets whole tables; no
    requests at all."""
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    table = torch.full((2, 6), -1, dtype=torch.int32, device=dev)
    t = pca.build_block_tables(table, i(0, 0), i(40, 20), i(*range(10, 20)), i(0), block_size=16, tokens=7)
    assert t.slots.tolist() == [160 + x for x in range(7)]
    assert table.tolist() == [[10, 11, 12, -1, -1, -1], [13, 14, -1, -1, -1, -1]]
    assert t.free_head.tolist() == [5] and t.q_start.tolist() == [0, 40, 60]
    t = pca.build_block_tables(table[:0], i(), i(), i(4), i(0), block_size=16, tokens=3)
    assert t.slots.tolist() == [-1] * 3 and t.q_start.tolist() == [0] and t.free_head.tolist() == [0]


# ---------------------------------------------------------------- together

def test_graph_replay(dev):
    """A decoding step captured in a HIP graph: tables, append, attention and a
    linear layer replay with new contents of the same buffers, and each replay
    equals the eager step."""
    rng = np.random.default_rng(21)
    heads, kv, dim, block, n = 8, 2, 64, 16, 3
    hidden = heads * dim
    layer, *_ = make_linear(rng, hidden, hidden, 64, False, False)

    def fresh():
        cache = pca.KV4Cache(200, block, kv, dim, group=32)
        return cache, torch.full((n, 60), -1, dtype=torch.int32, device=dev)

    lens0 = torch.tensor([0, 700, 33], dtype=torch.int32, device=dev)
    ones = torch.ones(n, dtype=torch.int32, device=dev)
    free = torch.arange(200, dtype=torch.int32, device=dev).flip(0).contiguous()
    data = [[torch.randn(n, h, dim, device=dev).bfloat16() for h in (heads, kv, kv)] for _ in range(5)]
    prefix = torch.randn(733, kv, dim, device=dev).bfloat16()

    def start(cache, table):
        t = pca.build_block_tables(table, torch.zeros_like(lens0), lens0, free, torch.zeros_like(ones[:1]),
                                   block_size=block, tokens=733)
        cache.append(prefix, prefix, t.slots)
        return t.context_lens.clone(), t.free_head.clone()

    def step(cache, table, lens, head, q, k, v):
        t = pca.build_block_tables(table, lens, ones, free, head, block_size=block, tokens=n)
        cache.append(k, v, t.slots)
        o = cache.attention(q, table, t.context_lens)
        y = layer.forward(o.view(n, hidden))
        lens.copy_(t.context_lens)
        head.copy_(t.free_head)
        return y

    cache, table = fresh()
    lens, head = start(cache, table)
    eager = [step(cache, table, lens, head, *d).clone() for d in data]

    cache, table = fresh()
    lens, head = start(cache, table)
    bufs = [b.clone() for b in data[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache, table, lens, head, *bufs)  # warm up
    torch.cuda.current_stream().wait_stream(side)
    cache.pool.zero_()
    table.fill_(-1)
    l0, h0 = start(cache, table)
    lens.copy_(l0)
    head.copy_(h0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(cache, table, lens, head, *bufs)
    for d, want in zip(data, eager):
        for b, x in zip(bufs, d):
            b.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        float(torch.randn(1000, device=dev).sum())  # eager work between the replays
