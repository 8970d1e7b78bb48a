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
