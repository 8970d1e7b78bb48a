"""Microscaled layers at the limits of their sizes and arguments: what the host
refuses before anything is launched, and the largest calls that it takes."""

import numpy as np
import pytest
import torch

import mx4_reference as ref
import popcount_convolution_amd as pca

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pca.load_library()
    return torch.device("cuda:0")


def make_experts(experts, k, n, seed=0):
    codes, scales = ref.random_weights(np.random.default_rng(seed), experts * n, k)
    codes, scales = codes.reshape(experts, n, -1), scales.reshape(experts, n, -1)
    return pca.MX4Experts(experts=experts, in_features=k, out_features=n, codes=codes, scales=scales), codes, scales


X, Y, OFFSETS, ORDER = 1 << 20, 2 << 20, 3 << 20, 4 << 20  # addresses that are never touched


@pytest.mark.parametrize("experts", [1, 3])
@pytest.mark.parametrize("x_rows,choices", [(1, 0x7fffffff), (1, (1 << 27) + 1), (1 << 14, (1 << 17) - 1), (3, 1 << 26)])
def test_more_rows_than_can_be_sorted(dev, experts, x_rows, choices):
    """Rows of experts are no more than the pairs that a sort takes: counts of
    them and of their blocks stay below 2^31."""
    layer, _, _ = make_experts(experts, 64, 16)
    args = pca.bconv_mx4_rows_t(X, 64, None, None, Y, 16, x_rows, x_rows * choices, pca.BCONV_BF16, choices, OFFSETS, ORDER)
    for call in (lambda: pca.bconv_mx4_linear_workspace_size(layer.handle, args),
                 lambda: pca.bconv_mx4_linear_forward(layer.handle, None, args)):
        with pytest.raises(pca.BconvError, match="more than 2\\^27") as e:
            call()
        assert e.value.status == pca.BCONV_ERR_INVALID_ARGUMENT
    args.rows, args.choices, args.x_rows = 1 << 27, 1 << 27, 1
    assert pca.bconv_mx4_linear_workspace_size(layer.handle, args) > 1 << 24  # the list of 2^20 row blocks


def test_most_input_rows(dev):
    """2^32 input values, as many as a layer of experts takes: the last codes end
    at byte 2^31 of the quantised rows, and the last row has its large values there."""
    tokens, k, n = 1 << 20, 4096, 20
    layer, codes, scales = make_experts(2, k, n)
    x = torch.randn((tokens, k), device=dev, dtype=torch.bfloat16)
    x[-1, -8:] = 500 + 100 * torch.arange(8, device=dev)
    ids = torch.zeros((tokens, 1), dtype=torch.int32, device=dev)
    ids[::3] = 1
    order = pca.sort_by_expert(ids, 2)
    q = pca.mx4_quantize(x)
    assert q.codes.numel() == 1 << 31
    y = layer.forward(q, order, dtype=torch.float32)
    assert torch.equal(layer.forward(x, order), y.to(torch.bfloat16))
    at = order.position[-40:, 0].long()
    rows, got = x[-40:].to(torch.float64).cpu().numpy(), y[at].to(torch.float64).cpu().numpy()
    for e in range(2):
        mine = (ids[-40:, 0] == e).cpu().numpy()
        want, mass = ref.linear(rows[mine], codes[e], scales[e], None)
        ok = (np.abs(got[mine] - want) <= ref.linear_bound(want, mass, k, "f32")).all(1)
        assert ok.all(), np.nonzero(mine)[0][~ok] - 40


DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [1, 3, 40, 300])
def test_columns_of_one_buffer(dev, dtype, rows):
    """Inputs and results side by side in one buffer, in both orders, give what
    buffers of their own do; columns that share one element are refused."""
    k, n, gap = 200, 51, 3
    layer, _, _ = make_experts(2, k, n)
    codes, scales = ref.random_weights(np.random.default_rng(1), n, k)
    linear = pca.MX4Linear(in_features=k, out_features=n, codes=codes, scales=scales)
    ids = (torch.arange(rows, dtype=torch.int32, device=dev) % 2).view(rows, 1)
    order = pca.sort_by_expert(ids, 2)
    values = torch.randn((rows, k), device=dev).to(DT[dtype])
    forwards = (linear.forward, lambda x, out=None: layer.forward(x, order, out=out),
                lambda x, out=None: layer.forward(x, order, out=out, in_order=True))
    for forward in forwards:
        want = forward(values)
        for x0, y0 in ((0, k), (n, 0), (n + gap, 1), (1, k + gap)):
            buf = torch.full((rows, k + n + gap + 2), 7.0, device=dev, dtype=DT[dtype])
            x, y = buf[:, x0:x0 + k], buf[:, y0:y0 + n]
            x.copy_(values)
            forward(x, out=y)
            assert torch.equal(y, want) and torch.equal(x, values)
            rest = torch.ones(buf.shape[1], dtype=torch.bool, device=dev)
            rest[x0:x0 + k] = rest[y0:y0 + n] = False
            assert bool((buf[:, rest] == 7).all())
        buf = torch.zeros((rows + 1, k + n + 2), device=dev, dtype=DT[dtype])
        for x0, y0 in ((0, k - 1), (n, 1), (0, 0)):
            with pytest.raises(pca.BconvError, match="overlap"):
                forward(buf[:rows, x0:x0 + k], out=buf[:rows, y0:y0 + n])
        if rows > 1:
            # a result that ends in the next row's inputs; one of another stride between the inputs
            for stride, y0 in ((k + n + 2, k + 3), (n + 1, k)):
                with pytest.raises(pca.BconvError, match="overlap"):
                    forward(buf[:rows, :k], out=buf.as_strided((rows, n), (stride, 1), y0))


def test_columns_of_one_buffer_of_tokens(dev):
    """As many columns of results as inputs, for tokens with several experts each:
    more result rows than input rows, in the same columns' stride."""
    tokens, choices, k, n = 30, 3, 96, 40
    layer, _, _ = make_experts(4, k, n)
    ids = torch.randint(0, 4, (tokens, choices), device=dev)
    order = pca.sort_by_expert(ids, 4)
    buf = torch.zeros((tokens * choices, k + n), device=dev)
    buf[:tokens, :k] = torch.randn((tokens, k), device=dev)
    want = layer.forward(buf[:tokens, :k].contiguous(), order)
    x = buf[:tokens, :k].clone()
    layer.forward(buf[:tokens, :k], order, out=buf[:, k:])
    assert torch.equal(buf[:, k:], want) and torch.equal(buf[:tokens, :k], x) and not bool(buf[tokens:, :k].any())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("tokens,choices,k,n", [(1, 1, 64, 16), (3, 2, 5000, 40), (20, 4, 600, 70), (300, 2, 9000, 30), (700, 3, 300, 600)])
def test_workspace_of_the_size_that_is_asked_for(dev, dtype, tokens, choices, k, n):
    """workspace_bytes() is what calls need: as much gives the same results as none
    given, a byte less is refused."""
    layer, _, _ = make_experts(3, k, n)
    codes, scales = ref.random_weights(np.random.default_rng(1), n, k)
    linear = pca.MX4Linear(in_features=k, out_features=n, codes=codes, scales=scales)
    x = torch.randn((tokens, k), device=dev).to(DT[dtype])
    order = pca.sort_by_expert(torch.randint(0, 3, (tokens, choices), device=dev), 3)
    rows = order.gather(x)
    q, qr = pca.mx4_quantize(x), pca.mx4_quantize(rows)
    sizes = set()
    for need, forward in (
            (linear.workspace_bytes(tokens, DT[dtype]), lambda **a: linear.forward(x, **a)),
            (linear.workspace_bytes(tokens, DT[dtype], quantised=True), lambda **a: linear.forward(q, dtype=DT[dtype], **a)),
            (layer.workspace_bytes(tokens, choices, DT[dtype]), lambda **a: layer.forward(x, order, **a)),
            (layer.workspace_bytes(tokens, choices, DT[dtype], quantised=True),
             lambda **a: layer.forward(q, order, dtype=DT[dtype], **a)),
            (layer.workspace_bytes(tokens, choices, DT[dtype], in_order=True), lambda **a: layer.forward(rows, order, in_order=True, **a)),
            (layer.workspace_bytes(tokens, choices, DT[dtype], in_order=True, quantised=True),
             lambda **a: layer.forward(qr, order, in_order=True, dtype=DT[dtype], **a))):
        sizes.add(need)
        want = forward()
        ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=dev)
        assert torch.equal(forward(workspace=ws[:need]), want) and bool((ws[need:] == 255).all())
        if need:
            with pytest.raises(ValueError, match=f"{need - 1} bytes given, {need} needed"):
                forward(workspace=ws[:need - 1])
    assert (sizes == {0}) == (tokens == 1)


# ---------------------------------------------------------- the largest sizes

def check_some(y, x, codes, scales, bias, dtype, rows, outs):
    """The results of some rows and outputs."""
    got = y[rows][:, outs].to(torch.float64).cpu().numpy()
    want, mass = ref.linear(x[rows].to(torch.float64).cpu().numpy(), codes[outs], scales[outs], None if bias is None else bias[outs])
    assert (np.abs(got - want) <= ref.linear_bound(want, mass, x.shape[1], dtype)).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,k,n", [(1, 1 << 20, 16), (5, (1 << 20) - 1, 40), (20, 1 << 20, 33), (150, 1 << 20, 20), (1, 32, 1 << 20),
                                      (3, 300, (1 << 20) - 5), (40, 33, 1 << 20), (200, 257, 1 << 20)])
def test_widest_layers(dev, dtype, rows, k, n):
    rng = np.random.default_rng(rows)
    codes, scales = ref.random_weights(rng, n, k)
    bias = rng.normal(0, 1, n).astype(np.float32)
    layer = pca.MX4Linear(in_features=k, out_features=n, codes=codes, scales=scales, bias=bias)
    x = torch.randn((rows, k), device=dev).to(DT[dtype])
    y = layer.forward(x)
    some = np.unique(np.concatenate([[0, n - 1, n // 2], rng.integers(0, n, 50)]))
    check_some(y, x, codes, scales, bias, dtype, np.unique([0, rows // 2, rows - 1]), some)
    q = layer.forward(pca.mx4_quantize(x), dtype=DT[dtype])
    check_some(q, x, codes, scales, bias, dtype, np.unique([0, rows // 2, rows - 1]), some)


@pytest.mark.parametrize("tokens,choices,k,n", [(1, 1, 40, 33), (700, 3, 40, 33), (3000, 8, 70, 300)])
def test_most_experts(dev, tokens, choices, k, n):
    layer, codes, scales = make_experts(1024, k, n, 3)
    rng = np.random.default_rng(tokens)
    ids = np.where(rng.random((tokens, choices)) < 0.3, 1023, rng.integers(-1, 1025, (tokens, choices)))
    ids[0, 0] = 1023
    offsets, order, _ = ref.expert_order(ids, 1024)
    o = pca.sort_by_expert(torch.from_numpy(ids).to(dev), 1024)
    assert np.array_equal(o.offsets.cpu().numpy(), offsets)
    x = torch.randn((tokens, k), device=dev)
    y, xs = layer.forward(x, o).to(torch.float64).cpu().numpy(), x.to(torch.float64).cpu().numpy()[np.maximum(order, 0) // choices]
    for e in range(1024):
        part = slice(offsets[e], offsets[e + 1])
        want, mass = ref.linear(xs[part], codes[e], scales[e], None)
        assert (np.abs(y[part] - want) <= ref.linear_bound(want, mass, k, "f32")).all(), e
    assert not y[offsets[-1]:].any()


@pytest.mark.parametrize("dtype", list(DT))
def test_quantise_in_slices(dev, dtype):
    """More rows than one launch quantises."""
    rows, cols = (1 << 25) + 3, 3
    x = torch.randn((rows, cols), device=dev).to(DT[dtype])
    q, values = pca.mx4_quantize(x, values=True)
    for part in (slice(0, 40), slice((1 << 25) - 40, rows), slice(12345678, 12345700)):
        codes, scales, want = ref.quantise(x[part].to(torch.float64).cpu().numpy())
        assert np.array_equal(q.codes[part].cpu().numpy(), codes) and np.array_equal(q.scales[part].cpu().numpy(), scales)
        assert np.array_equal(values[part].to(torch.float64).cpu().numpy(), want)
    # a value of fewer bits than it was made of stays what it is when it is quantised again
    assert torch.equal(pca.mx4_quantize(values, values=True)[1], values)


@pytest.mark.parametrize("choices", [1, 8])
def test_most_pairs(dev, choices):
    """2^27 pairs sorted, and rows of one value moved there and back."""
    tokens, experts = (1 << 27) // choices, 7
    ids = torch.randint(-1, experts, (tokens, choices), dtype=torch.int32, device=dev)
    o = pca.sort_by_expert(ids, experts)
    flat = ids.view(-1)
    key = torch.where(flat < 0, experts, flat)
    want = torch.sort(key.to(torch.int16), stable=True)[1].to(torch.int32)
    counts = torch.bincount(key, minlength=experts + 1)
    offsets = torch.cumsum(counts, 0) - counts
    assert torch.equal(o.offsets.long(), offsets)
    kept = int(offsets[-1])
    assert torch.equal(o.order[:kept], want[:kept]) and bool((o.order[kept:] == -1).all())
    del key, counts
    position = o.position.view(-1)
    assert bool((position[flat < 0] == -1).all())
    assert torch.equal(position[want[:kept].long()], torch.arange(kept, dtype=torch.int32, device=dev))
    x = torch.randint(-8, 9, (tokens, 1), device=dev).to(torch.bfloat16)
    rows = o.gather(x)
    assert torch.equal(rows[:kept, 0], x[want[:kept].long() // choices, 0]) and not bool(rows[kept:].any())
    times = (ids >= 0).sum(1, keepdim=True)
    assert torch.equal(o.combine(rows), (x.float() * times).to(torch.bfloat16))  # whole numbers up to 64
    d_rows, d_weights = o.combine_backward(x, rows, (ids >= 0).to(torch.bfloat16))
    assert torch.equal(d_rows, rows)
    assert torch.equal(d_weights, torch.where(ids >= 0, x.float() ** 2, 0).to(torch.bfloat16))


@pytest.mark.parametrize("tokens,choices", [(1, 3), (130, 2), (3, 1)])
def test_widest_rows(dev, tokens, choices):
    width = 1 << 20
    ids = torch.randint(0, 3, (tokens, choices), device=dev)
    ids[-1, 0] = 5
    o = pca.sort_by_expert(ids, 3)
    x = torch.randint(-4, 5, (tokens, width), device=dev).to(torch.float16)
    rows = o.gather(x)
    order = o.order.long()
    assert torch.equal(rows, torch.where((order >= 0)[:, None], x[order.clamp(min=0) // choices], 0))
    times = (ids < 3).sum(1, keepdim=True)
    assert torch.equal(o.combine(rows), x * times)
    weights = torch.randint(-2, 3, (tokens, choices), device=dev).float()
    d_rows, d_weights = o.combine_backward(x, rows, weights)
    assert torch.equal(d_rows, torch.where((order >= 0)[:, None], x[order.clamp(min=0) // choices] * weights.view(-1)[order.clamp(min=0), None].half(), 0))
    # whole numbers up to 2^24: exact in fp32 in any order
    assert torch.equal(d_weights.double(), torch.where(ids < 3, (x.double() ** 2).sum(1, keepdim=True), 0.0))


# ----------------------------------------------------- powers of two at the ends

@pytest.mark.parametrize("rows", [1, 5, 40, 300])
@pytest.mark.parametrize("low,x_exponent", [(0, 110), (3, 118), (250, -149), (247, -120), (251, -127)])
def test_range_of_the_powers(dev, rows, low, x_exponent):
    """Weights' powers of 2^-127 up, times the largest x, and of 2^124 down, times
    subnormal ones: their products are ordinary numbers."""
    rng = np.random.default_rng(rows + low)
    k, n = 640, 70
    codes, scales = ref.random_weights(rng, n, k, low, low + 3)
    layer = pca.MX4Linear(in_features=k, out_features=n, codes=codes, scales=scales)
    x = torch.from_numpy(np.ldexp(rng.integers(-15, 16, (rows, k)).astype(np.float64), x_exponent).astype(np.float32)).to(dev)
    assert bool(x.isfinite().all())
    for y in (layer.forward(x), layer.forward(pca.mx4_quantize(x), dtype=torch.float32)):
        check_some(y, x, codes, scales, None, "f32", np.arange(rows), np.arange(n))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [1, 16, 17])
def test_few_rows_of_a_large_layer(dev, dtype, rows):
    """More than 128 MiB of codes: read once for up to 16 rows, from 17 on by the kernel of many rows."""
    k, n = 16640, 16400
    rng = np.random.default_rng(rows)
    codes, scales = ref.random_weights(rng, n, k)
    layer = pca.MX4Linear(in_features=k, out_features=n, codes=codes, scales=scales)
    x = torch.randn((rows, k), device=dev).to(DT[dtype])
    some = np.unique(np.concatenate([[0, n - 1], rng.integers(0, n, 50)]))
    for y in (layer.forward(x), layer.forward(pca.mx4_quantize(x), dtype=DT[dtype])):
        check_some(y, x, codes, scales, None, dtype, np.arange(rows), some)
