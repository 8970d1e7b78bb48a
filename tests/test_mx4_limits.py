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
