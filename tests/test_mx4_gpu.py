"""Microscaled 4-bit quantisation and products, and tokens to experts and back,
on the GPU against plain 64-bit references (mx4_reference.py), at the sizes,
strides, orders and values where they can go wrong."""

import numpy as np
import pytest
import torch

import mx4_reference as ref
import popcount_convolution_amd as pca

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TYPES = ["bf16", "f16", "f32"]


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


def same(a, b):
    """Equal everywhere, NaN at the same places."""
    return bool(((a == b) | (np.isnan(a) & np.isnan(b))).all())


def rows_of(rng, rows, cols, dev, dtype, stride=0, scale=1.0):
    """Normal rows with a few large channels; with a stride, a view that starts one element in."""
    x = rng.normal(0, scale, (rows, cols)) * (1 + 30 * (rng.random(cols) < 0.02))
    t = torch.from_numpy(x.astype(np.float32)).to(dev).to(DT[dtype])
    if not stride:
        return t
    wide = torch.full((rows, cols + stride), 3.0, device=dev, dtype=DT[dtype])
    wide[:, 1:cols + 1] = t
    return wide[:, 1:cols + 1]


# --------------------------------------------------------------- quantisation

def check_quantised(x, q, values=None):
    codes, scales, want = ref.quantise(host(x).reshape(-1, x.shape[-1]))
    assert np.array_equal(q.scales.cpu().numpy().reshape(scales.shape), scales)
    assert np.array_equal(q.codes.cpu().numpy().reshape(codes.shape), codes)
    if values is not None:
        assert values.dtype == x.dtype and values.shape == x.shape
        assert same(host(values).reshape(want.shape), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,stride", [
    (1, 1, 0), (1, 31, 0), (1, 32, 0), (1, 33, 0), (2, 255, 0), (3, 256, 0), (2, 257, 3), (5, 100, 8), (7, 1000, 0),
    (33, 520, 5), (128, 4096, 0), (257, 2048, 8), (1000, 96, 0), (65, 5003, 0)])
def test_quantise(dev, dtype, rows, cols, stride):
    say("quantise", dtype, rows, cols, stride)
    rng = np.random.default_rng(rows * 1009 + cols)
    x = rows_of(rng, rows, cols, dev, dtype, stride)
    q, values = pca.mx4_quantize(x, values=True)
    check_quantised(x, q, values)
    assert q.cols == cols and torch.equal(pca.mx4_quantize(x).codes, q.codes)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantise_every_exponent(dev, dtype):
    """Blocks whose largest value runs through every exponent of the type,
    subnormal ones too, with values on and next to every border."""
    finfo = torch.finfo(DT[dtype])
    rng = np.random.default_rng(5)
    low = {"f32": -149, "f16": -24, "bf16": -133}[dtype]
    rows = []
    for e in range(low, {"f32": 128, "f16": 16, "bf16": 128}[dtype]):
        for fraction in (1.0, 1.25, 1.5, 1.75, 2 - 2.0 ** -7):
            block = np.concatenate([[fraction], rng.integers(0, 33, 16) / 16.0 * rng.choice([-1, 1], 16),
                                    rng.uniform(-1, 1, 15) * fraction])
            rows.append(np.clip(np.ldexp(block, e), finfo.min, finfo.max))
    x = torch.from_numpy(np.array(rows).reshape(-1, 5 * 32)).to(dev).to(DT[dtype])
    x = torch.where(x.isfinite(), x, torch.zeros_like(x))
    near = torch.where(torch.from_numpy(rng.random(x.shape) < 0.3).to(dev), torch.nextafter(
        x.cpu(), torch.full_like(x.cpu(), float("inf"))).to(dev) if dtype != "bf16" else x, x)
    near = torch.where(near.isfinite(), near, x)
    q, values = pca.mx4_quantize(near, values=True)
    check_quantised(near, q, values)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantise_special(dev, dtype):
    """Zeros of both signs, NaN and infinities: a block of its own each."""
    x = torch.randn((4, 32 * 12 + 7), device=dev).to(DT[dtype])
    x[0, :64] = 0
    x[1, :32] = -0.0
    x[0, 70] = float("nan")
    x[1, 100] = float("inf")
    x[2, 32 * 12 + 6] = -float("inf")
    x[3, 129] = torch.finfo(DT[dtype]).max
    q, values = pca.mx4_quantize(x, values=True)
    check_quantised(x, q, values)
    assert int(values.isnan().sum()) == 32 + 32 + 7


def test_quantise_shapes(dev):
    x = torch.randn((3, 5, 300), device=dev, dtype=torch.bfloat16)
    q = pca.mx4_quantize(x)
    assert q.codes.shape == (3, 5, 256) and q.scales.shape == (3, 5, 16) and q.cols == 300
    check_quantised(x, q)
    empty = pca.mx4_quantize(x[:0])
    assert empty.codes.shape == (0, 5, 256)
    v = torch.randn(40, device=dev)
    check_quantised(v.view(1, -1), pca.mx4_quantize(v))


# --------------------------------------------------------------------- linear

def make_linear(rng, k, n, bias, low=118, high=122):
    codes, scales = ref.random_weights(rng, n, k, low, high)
    b = rng.normal(0, 1, n).astype(np.float32) if bias else None
    return pca.MX4Linear(in_features=k, out_features=n, codes=codes, scales=scales, bias=b), (codes, scales, b)


def check_product(y, x, weights, dtype):
    want, mass = ref.linear(host(x).reshape(-1, x.shape[-1]), *weights)
    bound = ref.linear_bound(want, mass, x.shape[-1], dtype)
    got = host(y).reshape(want.shape)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / bound)} of its bound"


LINEAR = [
    (1, 1, 1, False), (1, 8, 5, True), (1, 32, 16, False), (1, 512, 512, True), (1, 4096, 96, False), (1, 5000, 67, False),
    (2, 129, 31, False), (3, 127, 33, True), (4, 257, 16, True), (5, 1000, 130, True), (15, 100, 17, False), (16, 256, 64, True),
    (17, 300, 48, True), (32, 640, 80, False), (33, 1025, 65, False), (48, 384, 200, True), (64, 2048, 128, True),
    (65, 1111, 129, True), (130, 777, 257, True), (200, 1536, 300, False), (257, 520, 140, True), (520, 260, 530, False),
    (1, 9000, 1100, False), (20, 9001, 700, True), (100, 6000, 1000, False), (300, 8200, 260, True), (1000, 513, 1030, False),
    (2100, 300, 2049, True)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k,n,bias", LINEAR)
def test_linear(dev, dtype, rows, k, n, bias):
    say("mx4 linear", dtype, rows, k, n, bias)
    rng = np.random.default_rng(rows * 1000003 + k * 1009 + n)
    layer, weights = make_linear(rng, k, n, bias)
    x = rows_of(rng, rows, k, dev, dtype)
    y = layer.forward(x)
    assert y.dtype == x.dtype and y.shape == (rows, n)
    check_product(y, x, weights, dtype)
    # strided rows, a strided result and a given workspace change nothing
    wide = torch.zeros((rows, k + 3), device=dev, dtype=DT[dtype])
    wide[:, 1:k + 1] = x
    buf = torch.full((rows, n + 5), 7.0, device=dev, dtype=DT[dtype])
    ws = torch.full((1 << 27,), 0xff, dtype=torch.uint8, device=dev)
    layer.forward(wide[:, 1:k + 1], out=buf[:, 2:n + 2], workspace=ws)
    assert torch.equal(buf[:, 2:n + 2], y) and bool((buf[:, :2] == 7).all()) and bool((buf[:, n + 2:] == 7).all())
    # and neither does quantising first
    q = pca.mx4_quantize(x)
    assert torch.equal(layer.forward(q, dtype=DT[dtype]), y)
    layer.close()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k,n,bias", [
    (300, 9000, 3000, True),      # two row blocks and a short one, inputs split between workgroups
    (150, 5000, 5000, False),     # a last block of up to 32 rows
    (190, 4900, 5003, True),      # of up to 64
    (129, 6400, 8200, False),     # of one row
    (1100, 1030, 1111, True),     # workgroups enough without splitting
    (2600, 260, 4100, True),      # wide workgroups
    (2050, 1800, 2049, False), (4000, 100, 600, True), (700, 2304, 2300, False)])
def test_linear_many_rows(dev, dtype, rows, k, n, bias):
    """Products large enough for the many-row kernel: each shape of its
    workgroups, short last blocks, tiles past the outputs, steps of 1 to many."""
    test_linear(dev, dtype, rows, k, n, bias)


def test_linear_slabs(dev):
    """More rows than one set of launches takes."""
    rng = np.random.default_rng(4)
    layer, weights = make_linear(rng, 30, 20, True)
    rows = (1 << 18) + 77
    x = rows_of(rng, rows, 30, dev, "f16")
    y = layer.forward(x)
    for part in (slice(0, 300), slice((1 << 18) - 150, (1 << 18) + 77)):
        check_product(y[part], x[part], weights, "f16")
    assert torch.equal(layer.forward(x[1 << 18:]), y[1 << 18:])
    assert torch.equal(layer.forward(pca.mx4_quantize(x), dtype=torch.float16), y)


@pytest.mark.parametrize("rows", [1, 5, 40, 300])
def test_linear_range(dev, rows):
    """Blocks from 2^-100 to 2^100, times weights as far apart, whose products are ordinary numbers."""
    rng = np.random.default_rng(rows)
    k, n = 640, 70
    layer, weights = make_linear(rng, k, n, False, 30, 31)       # weights of 2^-97
    x = rows_of(rng, rows, k, dev, "f32") * 2.0 ** 90
    check_product(layer.forward(x), x, weights, "f32")
    layer, weights = make_linear(rng, k, n, False, 227, 228)     # 2^100
    x = rows_of(rng, rows, k, dev, "f32") * 2.0 ** -100
    x[:, 64:96] = 0
    check_product(layer.forward(x), x, weights, "f32")


@pytest.mark.parametrize("rows,k,n", [(1, 700, 90), (5, 700, 90), (40, 700, 90), (300, 700, 90), (600, 700, 1500)])
def test_linear_nan(dev, rows, k, n):
    """A NaN or an infinity makes its row NaN and no other; a NaN scale of the weights its output."""
    rng = np.random.default_rng(rows)
    codes, scales = ref.random_weights(rng, n, k)
    scales[17, 3] = 255
    layer = pca.MX4Linear(in_features=k, out_features=n, codes=codes, scales=scales)
    x = rows_of(rng, rows, k, dev, "bf16")
    y = layer.forward(x)
    assert bool(y[:, 17].isnan().all()) and int(y.isnan().sum()) == rows
    x[rows // 2, 650] = float("inf")
    y = layer.forward(x)
    assert bool(y[rows // 2].isnan().all()) and int(y.isnan().sum()) == rows + n - 1


def test_linear_shapes(dev):
    rng = np.random.default_rng(1)
    layer, weights = make_linear(rng, 96, 40, True)
    x = rows_of(rng, 12, 96, dev, "f16")
    y = layer.forward(x)
    assert torch.equal(layer.forward(x.view(3, 4, 96)), y.view(3, 4, 40))
    assert torch.equal(layer.forward(x[0]), y[0])
    assert layer.forward(x[:0]).shape == (0, 40)
    q = pca.mx4_quantize(x)
    part = layer.forward(pca.MX4Tensor(q.codes[3:], q.scales[3:], 96), dtype=torch.float16)
    assert torch.equal(part, y[3:])
    assert layer.forward(q).dtype == torch.bfloat16
    out = torch.empty((12, 40), device=dev)
    assert layer.forward(q, out=out) is out
    check_product(out, x, weights, "f32")


# -------------------------------------------------------------------- experts

def make_ids(rng, tokens, choices, experts, dropped=0.0, skew=0.0, dtype=np.int64):
    score = rng.normal(0, 1, (tokens, experts)) + skew * rng.normal(0, 1, experts)
    ids = np.argsort(-score, 1)[:, :choices] if choices <= experts else rng.integers(0, experts, (tokens, choices))
    ids = np.where(rng.random(ids.shape) < dropped, rng.choice([-1, experts, experts + 5, -100], ids.shape), ids)
    return ids.astype(dtype)


SORTS = [(1, 1, 1, 0.0), (1, 8, 8, 0.0), (5, 3, 4, 0.5), (32, 4, 64, 0.0), (32, 8, 256, 0.1), (100, 2, 1000, 0.0), (100, 2, 1024, 0.0),
         (511, 1, 7, 0.3), (513, 6, 13, 0.0), (1024, 8, 16, 0.0), (1025, 8, 16, 0.05), (3001, 4, 60, 1.0), (3001, 4, 60, 0.02),
         (20000, 6, 128, 0.0), (66000, 8, 1023, 0.2), (0, 4, 5, 0.0)]


@pytest.mark.parametrize("ids_type", [np.int32, np.int64])
@pytest.mark.parametrize("tokens,choices,experts,dropped", SORTS)
def test_sort(dev, ids_type, tokens, choices, experts, dropped):
    say("sort", tokens, choices, experts, dropped)
    rng = np.random.default_rng(tokens * 31 + experts)
    ids = make_ids(rng, tokens, choices, experts, dropped, dtype=ids_type)
    o = pca.sort_by_expert(torch.from_numpy(ids).to(dev), experts)
    for got, want in zip((o.offsets, o.order, o.position), ref.expert_order(ids, experts)):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), want)
    assert (o.tokens, o.choices, o.experts) == (tokens, choices, experts)


def test_sort_far_ids(dev):
    """64-bit ids whose low halves name an expert are no experts."""
    ids = torch.tensor([[1 << 32, 1], [(1 << 40) + 2, -(1 << 33)], [0, 3]], device=dev)
    o = pca.sort_by_expert(ids, 3)
    assert o.offsets.tolist() == [0, 1, 2, 2] and o.position.tolist() == [[-1, 1], [-1, -1], [0, -1]]
    assert o.order.tolist() == [4, 1, -1, -1, -1, -1]


def test_sort_one_expert(dev):
    ids = torch.full((9001, 1), 5, dtype=torch.int32, device=dev)
    o = pca.sort_by_expert(ids, 9)
    assert o.offsets.tolist() == [0] * 6 + [9001] * 4 and torch.equal(o.order, torch.arange(9001, dtype=torch.int32, device=dev))


ROWS = [(1, 1, 1, 1, 0.0), (3, 2, 4, 7, 0.5), (32, 8, 256, 512, 0.0), (50, 4, 16, 1000, 0.1), (17, 6, 13, 4096, 0.2),
        (300, 1, 5, 264, 0.0), (9, 20, 3, 65, 0.3), (5, 2, 8, 5003, 0.0), (40, 3, 6, 2056, 1.0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,choices,experts,width,dropped", ROWS)
def test_rows(dev, dtype, tokens, choices, experts, width, dropped):
    """Gather, combine and their gradients, dense and strided, with each type of weights."""
    say("rows", dtype, tokens, choices, experts, width, dropped)
    rng = np.random.default_rng(tokens * 77 + width)
    ids = make_ids(rng, tokens, choices, experts, dropped)
    _, order, position = ref.expert_order(ids, experts)
    o = pca.sort_by_expert(torch.from_numpy(ids).to(dev), experts)
    pairs, eps, least = tokens * choices, ref.HALF_STEP[dtype], ref.LEAST[dtype] / 2
    kept = position >= 0
    at = np.maximum(position, 0)
    for stride in (0, 5, 8):
        x = rows_of(rng, tokens, width, dev, dtype, stride)
        want = np.where(order[:, None] >= 0, host(x)[np.maximum(order, 0) // choices], 0)
        assert np.array_equal(host(o.gather(x)), want)
        rows = rows_of(rng, pairs, width, dev, dtype, stride)
        d = rows_of(rng, tokens, width, dev, dtype, stride)
        taken = np.where(kept[..., None], host(rows)[at], 0)           # [tokens, choices, width]
        for weight_dtype in TYPES if not stride else ["f32"]:
            w = torch.from_numpy(rng.normal(0, 1, (tokens, choices))).to(dev).to(DT[weight_dtype])
            wh = np.where(kept, host(w), 0)
            # one rounding of 2^-24 a term, then the result's
            terms = taken * wh[..., None]
            y = host(o.combine(rows, w))
            bound = choices * 2.0 ** -24 * np.abs(terms).sum(1) + eps * np.abs(terms.sum(1)) * (1 + 2.0 ** -20) + least
            assert (np.abs(y - terms.sum(1)) <= bound).all()
            d_rows, d_weights = o.combine_backward(d, rows, w)
            assert d_rows.dtype == DT[dtype] and d_weights.dtype == DT[weight_dtype]
            want = np.zeros((pairs, width))
            want[position[kept]] = (host(d)[:, None] * wh[..., None])[kept]
            # fp32 products are rounded once, to fp32, before the type's rounding
            assert (np.abs(host(d_rows) - want) <= (eps + 2.0 ** -24) * np.abs(want) * (1 + 2.0 ** -20) + least).all()
            assert not host(d_rows)[order < 0].any()
            products = host(d)[:, None] * taken
            # additions one after the other in a lane, then over 64 lanes and 4 waves
            bound = ((width // 256 + 16) * 2.0 ** -24 * np.abs(products).sum(-1)
                     + ref.HALF_STEP[weight_dtype] * np.abs(products.sum(-1)) * (1 + 2.0 ** -10) + ref.LEAST[weight_dtype])
            assert (np.abs(host(d_weights) - products.sum(-1)) <= bound).all()
        ones = host(o.gather_backward(rows))
        bound = choices * 2.0 ** -24 * np.abs(taken).sum(1) + eps * np.abs(taken.sum(1)) * (1 + 2.0 ** -20) + least
        assert (np.abs(ones - taken.sum(1)) <= bound).all()
        assert torch.equal(o.combine(rows), o.gather_backward(rows))
        d_rows, none = o.combine_backward(d, rows)
        assert none is None and torch.equal(d_rows, o.gather(d))


def test_gradients_by_differences(dev):
    """The gradients against central differences of the forward calls, which
    are linear in each argument: steps of 1 make no error but fp32's."""
    rng = np.random.default_rng(3)
    ids = make_ids(rng, 6, 2, 4, 0.2)
    o = pca.sort_by_expert(torch.from_numpy(ids).to(dev), 4)
    x, rows, w, dy = (torch.from_numpy(rng.integers(-8, 9, s).astype(np.float32)).to(dev)
                      for s in ((6, 9), (12, 9), (6, 2), (6, 9)))
    d_rows, d_weights = o.combine_backward(dy, rows, w)

    def loss(r, v):
        return float((o.combine(r, v) * dy).sum())

    for t, grad, f in ((rows, d_rows, lambda r: loss(r, w)), (w, d_weights, lambda v: loss(rows, v)),
                       (x, o.gather_backward(rows), lambda v: float((o.gather(v) * rows).sum()))):
        for i in range(t.numel()):
            step = torch.zeros_like(t).view(-1)
            step[i] = 1
            step = step.view_as(t)
            # small whole numbers: every sum here is exact in fp32
            assert (f(t + step) - f(t - step)) / 2 == float(grad.reshape(-1)[i])


def test_dropped_rows_are_not_read(dev):
    """NaN in rows that belong to no pair, and in the weights of dropped pairs, reaches nothing."""
    ids = torch.tensor([[0, -1], [7, 1]], device=dev)
    o = pca.sort_by_expert(ids, 2)
    rows = torch.ones((4, 40), device=dev)
    rows[2:] = float("nan")
    w = torch.tensor([[2.0, float("nan")], [float("nan"), 3.0]], device=dev)
    assert torch.equal(o.combine(rows, w), torch.tensor([[2.0], [3.0]], device=dev).expand(2, 40))
    d_rows, d_weights = o.combine_backward(torch.ones((2, 40), device=dev), rows, w)
    assert d_weights.tolist() == [[40.0, 0.0], [0.0, 40.0]]
    assert d_rows[:, 0].tolist() == [2.0, 3.0, 0.0, 0.0]


EXPERTS = [
    # tokens, choices, experts, k, n, bias, dropped, skew
    (1, 1, 1, 32, 16, False, 0.0, 0.0), (1, 4, 8, 512, 300, True, 0.0, 0.0), (3, 2, 64, 300, 70, False, 0.3, 0.0),
    (32, 4, 64, 256, 176, True, 0.0, 0.0), (40, 2, 3, 1000, 65, True, 0.1, 0.0), (100, 3, 5, 129, 500, False, 0.0, 1.0),
    (200, 1, 4, 700, 33, True, 0.0, 3.0), (333, 4, 8, 520, 130, True, 0.05, 0.0), (700, 6, 7, 260, 300, False, 0.0, 0.0),
    (1500, 2, 3, 1024, 513, True, 0.0, 2.0), (600, 8, 16, 257, 272, False, 1.0, 0.0), (130, 2, 200, 320, 48, True, 0.0, 0.0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,choices,experts,k,n,bias,dropped,skew", EXPERTS)
def test_experts(dev, dtype, tokens, choices, experts, k, n, bias, dropped, skew):
    say("experts", dtype, tokens, choices, experts, k, n, dropped, skew)
    rng = np.random.default_rng(tokens * 7919 + k)
    ids = make_ids(rng, tokens, choices, experts, dropped, skew)
    offsets, order, _ = ref.expert_order(ids, experts)
    codes, scales = ref.random_weights(rng, experts * n, k)
    codes, scales = codes.reshape(experts, n, -1), scales.reshape(experts, n, -1)
    b = rng.normal(0, 1, (experts, n)).astype(np.float32) if bias else None
    layer = pca.MX4Experts(experts=experts, in_features=k, out_features=n, codes=codes, scales=scales, bias=b)
    o = pca.sort_by_expert(torch.from_numpy(ids).to(dev), experts)
    x = rows_of(rng, tokens, k, dev, dtype)
    buf = torch.full((tokens * choices, n + 5), 7.0, device=dev, dtype=DT[dtype])
    y = layer.forward(x, o, out=buf[:, 2:n + 2])
    assert bool((buf[:, :2] == 7).all()) and bool((buf[:, n + 2:] == 7).all())
    sorted_x = o.gather(x)
    for e in range(experts):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            check_product(y[lo:hi], sorted_x[lo:hi], (codes[e], scales[e], None if b is None else b[e]), dtype)
    assert not bool(y[int(offsets[-1]):].any())
    # the same from gathered rows, from quantised ones, and from both
    assert torch.equal(layer.forward(sorted_x, o, in_order=True), y)
    assert torch.equal(layer.forward(pca.mx4_quantize(x), o, dtype=DT[dtype]), y)
    assert torch.equal(layer.forward(pca.mx4_quantize(sorted_x), o, in_order=True, dtype=DT[dtype]), y)
    layer.close()


def test_experts_like_one_layer(dev):
    """One expert that has every row gives what a linear layer gives."""
    rng = np.random.default_rng(8)
    codes, scales = ref.random_weights(rng, 100, 400)
    one = pca.MX4Linear(in_features=400, out_features=100, codes=codes, scales=scales)
    layer = pca.MX4Experts(experts=1, in_features=400, out_features=100, codes=codes[None], scales=scales[None])
    for rows in (1, 30, 400):
        x = rows_of(rng, rows, 400, dev, "f32")
        o = pca.sort_by_expert(torch.zeros((rows, 1), dtype=torch.int64, device=dev), 1)
        want, mass = ref.linear(host(x), codes, scales, None)
        assert (np.abs(host(layer.forward(x, o)) - host(one.forward(x))) <= 2 * ref.linear_bound(want, mass, 400, "f32")).all()


def test_experts_offsets_out_of_order(dev):
    """Offsets and an order that no sort has given stay inside the buffers."""
    rng = np.random.default_rng(1)
    codes, scales = ref.random_weights(rng, 6 * 40, 64)
    layer = pca.MX4Experts(experts=6, in_features=64, out_features=40, codes=codes.reshape(6, 40, -1),
                           scales=scales.reshape(6, 40, -1))
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    for tokens in (50, 700, 5000):
        pairs = 2 * tokens
        x = rows_of(rng, tokens, 64, dev, "bf16")
        order = torch.randint(-(1 << 30), 1 << 30, (pairs,), device=dev, dtype=torch.int32)
        position = torch.randint(-(1 << 30), 1 << 30, (tokens, 2), device=dev, dtype=torch.int32)
        o = pca.ExpertOrder(ints([0, pairs, -5, pairs + 99, 0, pairs, 7]), order, position, 6)
        buf = torch.full((pairs + 2, 40), 7.0, device=dev, dtype=torch.bfloat16)
        layer.forward(x, o, out=buf[1:-1])
        layer.forward(x.repeat(2, 1), o, out=buf[1:-1], in_order=True)
        o.combine(o.gather(x))
        torch.cuda.synchronize()
        assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())


@pytest.mark.parametrize("rows", [16, 100])
def test_experts_one_has_all(dev, rows):
    """Every token at the last of many experts: its rows are more than one pass of a workgroup takes."""
    rng = np.random.default_rng(rows)
    codes, scales = ref.random_weights(rng, 40 * 50, 320)
    codes, scales = codes.reshape(40, 50, -1), scales.reshape(40, 50, -1)
    layer = pca.MX4Experts(experts=40, in_features=320, out_features=50, codes=codes, scales=scales)
    x = rows_of(rng, rows, 320, dev, "f16")
    o = pca.sort_by_expert(torch.full((rows, 1), 39, dtype=torch.int32, device=dev), 40)
    check_product(layer.forward(x, o), x, (codes[39], scales[39], None), "f16")


def test_wrappers_refuse(dev):
    """What the wrappers check once tensors are on the GPU."""
    rng = np.random.default_rng(0)
    o = pca.sort_by_expert(torch.zeros((4, 2), dtype=torch.int32, device=dev), 3)
    x, rows, w = (torch.zeros(s, device=dev) for s in ((4, 10), (8, 10), (4, 2)))
    layer, _ = make_linear(rng, 64, 10, False)
    codes, scales = ref.random_weights(rng, 3 * 10, 64)
    experts = pca.MX4Experts(experts=3, in_features=64, out_features=10, codes=codes.reshape(3, 10, -1),
                             scales=scales.reshape(3, 10, -1))
    xs = torch.zeros((4, 64), device=dev, dtype=torch.bfloat16)
    q = pca.mx4_quantize(xs)
    for f, match in (
            (lambda: o.combine(rows, torch.zeros((8, 1), device=dev)), "shape"), (lambda: o.combine(rows, w.double()), "dtype"),
            (lambda: o.combine(rows, w.t().contiguous().t()), "contiguous"), (lambda: o.combine(rows, w.cpu()), "device"),
            (lambda: o.combine(rows, w, out=x[:, :9]), "shape"), (lambda: o.gather(x, out=rows.half()), "dtype"),
            (lambda: o.combine_backward(x, rows[:, :9], w), "values"), (lambda: o.combine_backward(x, rows.half(), w), "dtype"),
            (lambda: o.combine_backward(x, rows, None, d_weights=w), "without weights"), (lambda: o.gather(x.cpu()), "device"),
            (lambda: o.gather(torch.zeros((10, 4), device=dev).t()), "strides"),
            (lambda: layer.forward(xs[:, :63]), "does not end"), (lambda: layer.forward(xs.cpu()), "device"),
            (lambda: layer.forward(xs, out=torch.zeros((4, 11), device=dev)), "shape"),
            (lambda: layer.forward(xs, out=torch.zeros((4, 10), device=dev)), "dtype"),
            (lambda: layer.forward(xs, dtype=torch.float32), "their type"), (lambda: layer.forward(q, dtype=torch.int32), "dtype"),
            (lambda: layer.forward(pca.MX4Tensor(q.codes, q.scales, 60)), "rows of 60"),
            (lambda: layer.forward(pca.MX4Tensor(q.codes[:, :64], q.scales, 64)), "codes: shape|scales: shape"),
            (lambda: layer.forward(pca.MX4Tensor(q.codes, q.scales[:3], 64)), "scales: shape"),
            (lambda: layer.forward(torch.zeros((300, 64), device=dev, dtype=torch.bfloat16),
                                   workspace=torch.zeros(8, dtype=torch.uint8, device=dev)), "needed"),
            (lambda: experts.forward(xs, None), "ExpertOrder"), (lambda: experts.forward(xs[:3], o), "rows"),
            (lambda: experts.forward(xs, o, in_order=True), "rows"),
            (lambda: experts.forward(xs, pca.sort_by_expert(torch.zeros((4, 2), dtype=torch.int32, device=dev), 4)), "4 experts"),
            (lambda: pca.MX4Linear(in_features=64, out_features=10, codes=codes, scales=scales), "shape"),
            (lambda: pca.MX4Linear(in_features=64, out_features=30, codes=codes.astype(np.int8), scales=scales), "dtype"),
            (lambda: pca.MX4Linear(in_features=0, out_features=30, codes=codes, scales=scales), "positive"),
            (lambda: pca.sort_by_expert(torch.zeros((4, 2), dtype=torch.int32, device=dev), 0), "experts"),
            (lambda: pca.sort_by_expert(torch.zeros((4, 2), dtype=torch.int32, device=dev), 1025), "experts")):
        with pytest.raises(ValueError, match=match):
            f()
    for f in (lambda: o.combine(rows, out=rows[:4]),
              lambda: experts.forward(xs, o, out=xs.as_strided((8, 10), (32, 1)))):
        with pytest.raises(pca.BconvError, match="overlap"):
            f()


# -------------------------------------------------------------- far offsets

def test_rows_past_32_bits(dev):
    """Results of more than 2^32 bytes."""
    tokens, width = 70001, 32768
    x = torch.randn((2, width), device=dev).to(torch.bfloat16).repeat_interleave(torch.tensor([tokens - 1, 1], device=dev), 0)
    ids = torch.zeros((tokens, 1), dtype=torch.int32, device=dev)
    ids[0] = 1                                                       # the first token's row is the last
    o = pca.sort_by_expert(ids, 2)
    rows = o.gather(x)
    assert torch.equal(rows[-1], x[0]) and torch.equal(rows[-2], x[-1]) and torch.equal(rows[0], x[1])
    rows[-1] *= 2
    y = o.combine(rows)
    assert torch.equal(y[0], x[0] * 2) and torch.equal(y[-1], x[-1]) and torch.equal(y[-2], x[-2])
    del rows, y
    q, values = pca.mx4_quantize(x, values=True)
    want = ref.quantise(host(x[-2:]))
    assert np.array_equal(q.codes[-2:].cpu().numpy(), want[0]) and np.array_equal(host(values[-2:]), want[2])


def test_products_past_32_bits(dev):
    """Results, and codes of all experts, of more than 2^32 bytes."""
    rng = np.random.default_rng(9)
    layer, weights = make_linear(rng, 40, 32771, True)
    x = rows_of(rng, 66000, 40, dev, "f16")
    y = layer.forward(x)
    check_product(y[-130:], x[-130:], weights, "f16")
    check_product(y[:5], x[:5], weights, "f16")
    del y
    layer.close()
    experts, k, n = 130, 8192, 8200
    codes = torch.randint(0, 256, (experts, n, k // 2), dtype=torch.uint8, device=dev)
    scales = torch.randint(118, 122, (experts, n, k // 32), dtype=torch.uint8, device=dev)
    layer = pca.MX4Experts(experts=experts, in_features=k, out_features=n, codes=codes, scales=scales)
    for tokens in (2, 30):
        x = rows_of(rng, tokens, k, dev, "bf16")
        ids = torch.full((tokens, 100), experts - 1, dtype=torch.int32, device=dev)
        ids[:, 1:] = -1
        ids[0, 0] = 0
        o = pca.sort_by_expert(ids, experts)
        y = layer.forward(x, o)
        for e, part in ((0, slice(0, 1)), (experts - 1, slice(1, tokens))):
            w = codes[e].cpu().numpy(), scales[e].cpu().numpy(), None
            check_product(y[part], x[0:1] if e == 0 else x[1:], w, "bf16")


# --------------------------------------------------- together, streams, graphs

class Block:
    """A feed-forward layer of experts as a model would run it."""

    def __init__(self, rng, width, hidden, experts):
        def layer(n, k):
            codes, scales = ref.random_weights(rng, experts * n, k, 116, 119)
            w = codes.reshape(experts, n, -1), scales.reshape(experts, n, -1)
            return pca.MX4Experts(experts=experts, in_features=k, out_features=n, codes=w[0], scales=w[1]), w
        self.up, self.up_w = layer(2 * hidden, width)
        self.down, self.down_w = layer(width, hidden)
        self.hidden, self.experts = hidden, experts

    def __call__(self, x, ids, weights):
        order = pca.sort_by_expert(ids, self.experts)
        both = self.up.forward(x, order)
        h = torch.nn.functional.silu(both[:, :self.hidden]) * both[:, self.hidden:]
        rows = self.down.forward(h, order, in_order=True)
        return order, both, h, rows, order.combine(rows, weights)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens", [1, 30, 500])
def test_layer_of_experts(dev, dtype, tokens):
    """Each step of a layer from what the step before it gave."""
    rng = np.random.default_rng(tokens)
    width, hidden, experts, choices = 320, 288, 6, 3
    block = Block(rng, width, hidden, experts)
    ids = make_ids(rng, tokens, choices, experts, 0.1)
    offsets, order, position = ref.expert_order(ids, experts)
    x = rows_of(rng, tokens, width, dev, dtype)
    weights = torch.from_numpy(rng.random((tokens, choices)).astype(np.float32)).to(dev)
    o, both, h, rows, y = block(x, torch.from_numpy(ids).to(dev), weights)
    assert np.array_equal(o.position.cpu().numpy(), position)
    xs = np.where(order[:, None] >= 0, host(x)[np.maximum(order, 0) // choices], 0)
    for got, inputs, w in ((both, xs, block.up_w), (rows, host(h), block.down_w)):
        for e in range(experts):
            part = slice(offsets[e], offsets[e + 1])
            want, mass = ref.linear(inputs[part], w[0][e], w[1][e], None)
            assert (np.abs(host(got)[part] - want) <= ref.linear_bound(want, mass, inputs.shape[1], dtype)).all()
    assert not host(rows)[offsets[-1]:].any()
    terms = np.where((position >= 0)[..., None], host(rows)[np.maximum(position, 0)], 0) * host(weights)[..., None]
    bound = (choices * 2.0 ** -24 * np.abs(terms).sum(1) + ref.HALF_STEP[dtype] * np.abs(terms.sum(1)) * (1 + 2.0 ** -20)
             + ref.LEAST[dtype])
    assert (np.abs(host(y) - terms.sum(1)) <= bound).all()


@pytest.mark.parametrize("tokens", [3, 300])
def test_graph_replays(dev, tokens):
    """A captured layer with changing inputs, between eager work, and two
    captured graphs in turn."""
    rng = np.random.default_rng(tokens)
    block = Block(rng, 320, 288, 6)
    linear, _ = make_linear(rng, 6000, 3000, True)
    x = rows_of(rng, tokens, 320, dev, "bf16")
    wide = rows_of(rng, tokens, 6000, dev, "bf16")
    ids = torch.from_numpy(make_ids(rng, tokens, 3, 6, 0.1)).to(dev)
    weights = torch.rand((tokens, 3), device=dev)
    dy = rows_of(rng, tokens, 320, dev, "bf16")

    def run():
        o, _, _, rows, y = block(x, ids, weights)
        return [o.order.clone(), y, *o.combine_backward(dy, rows, weights), o.gather_backward(o.gather(x)), linear.forward(wide),
                pca.mx4_quantize(x, values=True)[1]]

    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    results = []
    for g in graphs:
        with torch.cuda.graph(g, stream=side):
            results.append(run())
    for turn in range(4):
        x.copy_(rows_of(rng, tokens, 320, dev, "bf16"))
        wide.copy_(rows_of(rng, tokens, 6000, dev, "bf16"))
        ids.copy_(torch.from_numpy(make_ids(rng, tokens, 3, 6, 0.2)).to(dev))
        want = run()
        for g in graphs if turn % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for got in results:
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_streams(dev):
    """Calls on another stream than the current one, two of them at once."""
    rng = np.random.default_rng(2)
    block = Block(rng, 320, 288, 6)
    linear, _ = make_linear(rng, 6000, 3000, True)
    ids = torch.from_numpy(make_ids(rng, 400, 2, 6)).to(dev)
    x, wide = rows_of(rng, 400, 320, dev, "bf16"), rows_of(rng, 400, 6000, dev, "bf16")
    want = pca.sort_by_expert(ids, 6)
    up, y, q = block.up.forward(x, want), linear.forward(wide), pca.mx4_quantize(wide)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams * 3:
        o = pca.sort_by_expert(ids, 6, stream=s)
        got.append((o.order, block.up.forward(x, o, stream=s), linear.forward(wide, stream=s),
                    pca.mx4_quantize(wide, stream=s).codes, o.combine(o.gather(x, stream=s), stream=s)))
    torch.cuda.synchronize()
    for order, u, v, codes, back in got:
        assert torch.equal(order, want.order) and torch.equal(u, up) and torch.equal(v, y) and torch.equal(codes, q.codes)
        assert torch.equal(back, want.combine(want.gather(x)))


def test_results_repeat(dev):
    """Bit for bit: no sum depends on an order that changes."""
    rng = np.random.default_rng(6)
    block = Block(rng, 320, 288, 6)
    x = rows_of(rng, 700, 320, dev, "f32")
    ids = torch.from_numpy(make_ids(rng, 700, 4, 6, 0.1)).to(dev)
    weights = torch.rand((700, 4), device=dev)
    first = block(x, ids, weights)
    grads = first[0].combine_backward(x, first[3], weights)
    for _ in range(3):
        again = block(x, ids, weights)
        for a, b in zip((*first[1:], *grads), (*again[1:], *again[0].combine_backward(x, again[3], weights))):
            assert torch.equal(a, b)
