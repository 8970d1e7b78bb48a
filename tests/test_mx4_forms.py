"""The forms of the kernels of layers of experts that sizes choose between, each
against plain 64-bit references (mx4_reference.py): gradients of several choices a
workgroup, rows stored past the caches, wide workgroups with lists of row blocks."""

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


def make_ids(rng, tokens, choices, experts, dropped):
    ids = rng.integers(0, experts, (tokens, choices))
    return np.where(rng.random(ids.shape) < dropped, rng.choice([-1, experts, experts + 5], ids.shape), ids)


def random(shape, dev, dtype, seed, pad=0):
    """Normal values; with `pad`, a view of rows that are that much further apart."""
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn((shape[0], shape[1] + pad), generator=g, device=dev).to(DT[dtype])[:, :shape[1]]


def check_rows(dev, dtype, tokens, choices, experts, width, dropped, weight_dtype, pad):
    """Gather, combine and both gradients; sums in 64 bits on the GPU."""
    rng = np.random.default_rng(tokens * 131 + choices * 17 + width)
    ids = make_ids(rng, tokens, choices, experts, dropped)
    _, order, position = ref.expert_order(ids, experts)
    o = pca.sort_by_expert(torch.from_numpy(ids).to(dev), experts)
    assert np.array_equal(o.position.cpu().numpy(), position)
    order, position = torch.from_numpy(order).to(dev).long(), torch.from_numpy(position).to(dev).long()
    pairs, eps, least = tokens * choices, ref.HALF_STEP[dtype], ref.LEAST[dtype] / 2
    kept, used = position >= 0, order >= 0
    x, rows, dy = (random((n, width), dev, dtype, i, pad) for i, n in enumerate((tokens, pairs, tokens)))
    w = random((tokens, choices), dev, weight_dtype, 3).contiguous()
    ones = torch.ones_like(w)

    got = o.gather(x)
    assert torch.equal(got[used], x[order[used] // choices]) and not bool(got[~used].any())
    del got

    def check_sum(y, factors):
        # one rounding of 2^-24 a term, then the result's
        total = torch.zeros((tokens, width), dtype=torch.float64, device=dev)
        mass = torch.zeros_like(total)
        for j in range(choices):
            part = rows[position[:, j].clamp(min=0)].double() * torch.where(kept[:, j], factors[:, j].double(), 0)[:, None]
            total += part
            mass += part.abs()
        bound = choices * 2.0 ** -24 * mass + eps * total.abs() * (1 + 2.0 ** -20) + least
        assert y.dtype == DT[dtype] and bool(((y.double() - total).abs() <= bound).all())

    check_sum(o.combine(rows, w), w)
    check_sum(o.combine(rows), ones)
    check_sum(o.gather_backward(rows), ones)

    d_rows, d_weights = o.combine_backward(dy, rows, w)
    plain, none = o.combine_backward(dy, None)
    assert none is None and d_weights.dtype == DT[weight_dtype]
    assert not bool(d_rows[~used].any()) and not bool(plain[~used].any())
    for j in range(choices):
        have, at = kept[:, j], position[:, j][kept[:, j]]
        d, r, f = dy[have].double(), rows[at].double(), w[have, j].double()
        # the fp32 product is rounded once before the type's rounding
        want = d * f[:, None]
        assert bool(((d_rows[at].double() - want).abs() <= (eps + 2.0 ** -24) * want.abs() * (1 + 2.0 ** -20) + least).all())
        assert torch.equal(plain[at], dy[have])
        # a lane's additions one after the other, then over 64 lanes and 4 waves
        products = d * r
        bound = ((width // 256 + 16) * 2.0 ** -24 * products.abs().sum(1)
                 + ref.HALF_STEP[weight_dtype] * products.sum(1).abs() * (1 + 2.0 ** -10) + ref.LEAST[weight_dtype])
        assert bool(((d_weights[have, j].double() - products.sum(1)).abs() <= bound).all())
        assert not bool(d_weights[~have, j].any())


# More tokens than share a workgroup's row: one takes all choices, in steps of eight,
# and its waves' sums of a step are in the same place as the next step's.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,choices,experts,width,dropped", [
    (129, 2, 4, 7, 0.2), (200, 4, 16, 1000, 0.1), (150, 8, 13, 264, 0.0), (150, 11, 13, 520, 0.2), (131, 17, 5, 2056, 0.1),
    (300, 6, 8, 5003, 0.3), (128, 9, 20, 777, 0.1), (129, 16, 20, 1, 0.5), (140, 24, 3, 4096, 1.0)])
def test_several_choices_a_workgroup(dev, dtype, tokens, choices, experts, width, dropped):
    for weight_dtype in TYPES:
        say("rows", dtype, tokens, choices, experts, width, dropped, weight_dtype)
        check_rows(dev, dtype, tokens, choices, experts, width, dropped, weight_dtype, 3 if weight_dtype == dtype else 0)


# Rows of more than 64 MiB: stored past the caches.
@pytest.mark.parametrize("dtype,tokens,choices,experts,width,dropped,weight_dtype,pad", [
    ("bf16", 2051, 5, 8, 4096, 0.1, "f32", 0), ("f16", 1025, 9, 16, 4160, 0.05, "f16", 8), ("f32", 701, 6, 7, 5003, 0.1, "f32", 0),
    ("bf16", 1500, 8, 16, 3333, 0.02, "bf16", 5), ("f32", 513, 11, 9, 3104, 0.3, "bf16", 0), ("f16", 100, 40, 9, 9001, 0.1, "f32", 0)])
def test_rows_past_the_caches(dev, dtype, tokens, choices, experts, width, dropped, weight_dtype, pad):
    say("rows past the caches", dtype, tokens, choices, experts, width, dropped, weight_dtype, pad)
    assert tokens * choices * width * (4 if dtype == "f32" else 2) > 1 << 26
    check_rows(dev, dtype, tokens, choices, experts, width, dropped, weight_dtype, pad)


def make_experts(rng, experts, k, n, bias):
    codes, scales = ref.random_weights(rng, experts * n, k)
    codes, scales = codes.reshape(experts, n, -1), scales.reshape(experts, n, -1)
    b = rng.normal(0, 1, (experts, n)).astype(np.float32) if bias else None
    layer = pca.MX4Experts(experts=experts, in_features=k, out_features=n, codes=codes, scales=scales, bias=b)
    return layer, codes, scales, b


# Rows of each expert: none, one, up to 32, 64 and 128, a whole block of 128 and
# its neighbours, several blocks, more than the 16 that are taken together.
COUNTS = [0, 1, 2, 17, 31, 32, 33, 50, 64, 65, 100, 127, 128, 129, 160, 193, 256, 300, 385, 2100]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k,n,bias,dropped", [
    (300, 4000, True, 37),     # wide workgroups: as many as there are compute units
    (1100, 2100, False, 0), (70, 8200, True, 1),
    (520, 130, True, 200)])    # narrow ones
def test_row_blocks_of_every_size(dev, dtype, k, n, bias, dropped):
    say("row blocks", dtype, k, n, bias, dropped)
    rng = np.random.default_rng(k + n)
    experts = len(COUNTS)
    layer, codes, scales, b = make_experts(rng, experts, k, n, bias)
    counts = rng.permutation(COUNTS)
    flat = np.concatenate([np.repeat(np.arange(experts), counts), np.full(dropped, -1)])
    rng.shuffle(flat)
    choices = 3 if flat.size % 3 == 0 else 2 if flat.size % 2 == 0 else 1
    tokens = flat.size // choices
    blocks = -(-flat.size // 128) + experts + 1
    cus = torch.cuda.get_device_properties(dev).multi_processor_count
    assert (blocks * -(-n // 256) >= cus) == (n >= 2000)
    ids = flat.reshape(tokens, choices)
    offsets, order, _ = ref.expert_order(ids, experts)
    o = pca.sort_by_expert(torch.from_numpy(ids).to(dev), experts)
    x = random((tokens, k), dev, dtype, 5, 3)
    buf = torch.full((flat.size, n + 5), 7.0, device=dev, dtype=DT[dtype])
    y = layer.forward(x, o, out=buf[:, 2:n + 2])
    assert bool((buf[:, :2] == 7).all()) and bool((buf[:, n + 2:] == 7).all())
    assert not bool(y[int(offsets[-1]):].any())
    xs = host(x)[np.maximum(order, 0) // choices]
    for e in range(experts):
        part = slice(offsets[e], offsets[e + 1])
        if offsets[e + 1] > offsets[e]:
            want, mass = ref.linear(xs[part], codes[e], scales[e], None if b is None else b[e])
            ok = np.abs(host(y[part]) - want) <= ref.linear_bound(want, mass, k, dtype)
            assert ok.all(), (e, counts[e], np.argwhere(~ok)[:3])
    gathered = o.gather(x)
    assert torch.equal(layer.forward(gathered, o, in_order=True), y)
    assert torch.equal(layer.forward(pca.mx4_quantize(x), o, dtype=DT[dtype]), y)
    assert torch.equal(layer.forward(pca.mx4_quantize(gathered), o, in_order=True, dtype=DT[dtype]), y)


@pytest.mark.parametrize("counts", [(0, 0, 0), (0, 5, 0), (3, 0, 4)])
def test_order_is_checked(dev, counts):
    """Tensors of an order on the GPU, each with one thing wrong; a right one works."""
    flat = np.repeat(np.arange(3), counts)
    if flat.size % 2:
        flat = np.append(flat, -1)
    tokens = flat.size // 2
    offsets, order, position = (torch.from_numpy(a).to(dev) for a in ref.expert_order(flat.reshape(tokens, 2), 3))
    x = torch.arange(tokens, device=dev, dtype=torch.float32).view(tokens, 1).expand(tokens, 5).contiguous()
    got = pca.ExpertOrder(offsets, order, position, 3).gather(x)
    assert torch.equal(got, torch.where((order >= 0)[:, None], x[order.clamp(min=0) // 2] if tokens else got, 0.0))
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    for bad, match in (
            ((ints(3), order, position), "^offsets: shape \\(3,\\) != \\(4,\\)"), ((offsets.long(), order, position), "^offsets: dtype"),
            ((ints(8)[::2], order, position), "^offsets: .*contiguous"), ((offsets.cpu(), order, position), "^offsets: .*device"),
            ((offsets, ints(2 * tokens + 1), position), "^order: shape"), ((offsets, order.long(), position), "^order: dtype"),
            ((offsets, order, ints(2 * tokens)), "^position: shape"), ((offsets, order, position.long()), "^position: dtype"),
            ((offsets, order, ints(tokens, 0)), "^position: shape"), ((offsets, order, None), "^position: a torch tensor"),
            ((None, order, position), "^offsets: a torch tensor"), ((offsets, None, position), "^order: a torch tensor")):
        with pytest.raises(ValueError, match=match):
            pca.ExpertOrder(*bad, 3)
    if tokens > 1:
        for bad, match in (((offsets, ints(4 * tokens)[::2], position), "^order: .*contiguous"),
                           ((offsets, order.cpu(), position), "^order: .*device"),
                           ((offsets, order, ints(2, tokens).t()), "^position: .*contiguous"),
                           ((offsets, order, position.cpu()), "on cuda:0, not on cpu|^position: .*device")):
            with pytest.raises(ValueError, match=match):
                pca.ExpertOrder(*bad, 3)


# Rows quantised in the products and in a launch before them, a few of each expert.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("experts,each,k,n", [
    (8, 12, 500, 300), (8, 13, 500, 300), (5, 8, 2048, 260), (5, 9, 2048, 260), (16, 3, 2304, 70), (16, 3, 2305, 70),
    (6, 12, 1281, 1030), (128, 2, 1024, 256), (128, 2, 1030, 272), (64, 2, 2000, 1030), (3, 16, 257, 2100)])
def test_few_rows_of_each_expert(dev, dtype, experts, each, k, n):
    say("few rows each", dtype, experts, each, k, n)
    rng = np.random.default_rng(experts * each + k)
    layer, codes, scales, b = make_experts(rng, experts, k, n, True)
    counts = rng.multinomial(experts * each, np.ones(experts) / experts)
    flat = rng.permutation(np.repeat(np.arange(experts), counts))
    choices = 2 if flat.size % 2 == 0 else 1
    ids = flat.reshape(-1, choices)
    offsets, order, _ = ref.expert_order(ids, experts)
    o = pca.sort_by_expert(torch.from_numpy(ids).to(dev), experts)
    x = random((ids.shape[0], k), dev, dtype, 7, 1)
    y = layer.forward(x, o)
    xs = host(x)[order // choices]
    for e in range(experts):
        part = slice(offsets[e], offsets[e + 1])
        want, mass = ref.linear(xs[part], codes[e], scales[e], b[e])
        assert (np.abs(host(y[part]) - want) <= ref.linear_bound(want, mass, k, dtype)).all(), e
    assert torch.equal(layer.forward(pca.mx4_quantize(x), o, dtype=DT[dtype]), y)
    assert torch.equal(layer.forward(o.gather(x), o, in_order=True), y)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k,n", [
    (1, 3328, 300), (1, 3329, 300), (1, 5120, 300), (1, 5121, 300), (12, 2048, 70), (13, 2048, 70), (8, 5120, 50), (8, 5121, 50),
    (7, 3300, 8300), (16, 1500, 8300), (16, 2600, 8300), (2, 2048, 16411)])
def test_few_rows_of_one_layer(dev, dtype, rows, k, n):
    say("few rows", dtype, rows, k, n)
    rng = np.random.default_rng(rows * 7 + k)
    codes, scales = ref.random_weights(rng, n, k)
    b = rng.normal(0, 1, n).astype(np.float32)
    layer = pca.MX4Linear(in_features=k, out_features=n, codes=codes, scales=scales, bias=b)
    x = random((rows, k), dev, dtype, 8, 1)
    want, mass = ref.linear(host(x), codes, scales, b)
    bound = ref.linear_bound(want, mass, k, dtype)
    assert (np.abs(host(layer.forward(x)) - want) <= bound).all()
    # from quantised rows the inputs may be split between other numbers of waves
    assert (np.abs(host(layer.forward(pca.mx4_quantize(x), dtype=DT[dtype])) - want) <= bound).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k,n", [(1, 300, 16384), (3, 300, 16385), (16, 40, 16400), (9, 2049, 16400)])
def test_few_rows_of_many_outputs(dev, dtype, rows, k, n):
    """Around as many outputs as compute units take at once, from where on rows are quantised in a launch."""
    test_few_rows_of_one_layer(dev, dtype, rows, k, n)
