"""The example of a layer of experts (examples/mx4_experts.py): it runs, and the
router's gradient is that of its formula and of differences."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def test_runs(dev):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "mx4_experts.py"), "--tokens", "33", "--width", "320",
                        "--hidden", "200", "--experts", "5", "--choices", "2"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr
    assert "33 tokens, 2 of 5 experts" in r.stdout


def test_router_gradient(dev):
    import mx4_experts
    layer = mx4_experts.ExpertLayer(96, 64, 6, 3, seed=1, dtype=torch.float32)
    x = torch.randn((20, 96), device=dev)
    y, saved = layer.forward(x)
    dy = torch.randn_like(y)
    grad = layer.router_gradient(dy, saved).double().cpu().numpy()
    _, ids, weights, order, rows = saved
    position = order.position.long()
    taken = rows[position].double()                                     # [tokens, choices, width]
    router = layer.router.double()
    logits = (x.double() @ router.t()).gather(1, ids)

    def loss(z):
        return ((torch.softmax(z, 1)[..., None] * taken).sum(1) * dy.double()).sum()

    # the same sums in 64 bits: fp32 makes at most a few roundings a term
    products = (taken * dy.double()[:, None]).sum(-1)
    w = torch.softmax(logits, 1)
    d_logits = w * (products - (w * products).sum(1, keepdim=True))
    want, mass = np.zeros_like(grad), np.zeros_like(grad)
    size = (w * (taken.abs() * dy.double().abs()[:, None]).sum(-1)).sum(1)
    for t in range(20):
        for j in range(3):
            want[ids[t, j].item()] += (d_logits[t, j] * x[t].double()).cpu().numpy()
            mass[ids[t, j].item()] += (size[t] * x[t].abs().double()).cpu().numpy()
    # sums of 96 products, of 96 logit terms that weights depend on, of 3 and of 20 rows
    assert (np.abs(grad - want) <= 2 * (96 + 96 * 4 + 3 + 20) * 2.0 ** -24 * mass + 1e-30).all()
    # central differences of the loss in a logit: the error of the difference is of the third order
    step = 1e-4
    for t, j in ((0, 0), (7, 2), (19, 1)):
        e = torch.zeros_like(logits)
        e[t, j] = step
        difference = (loss(logits + e) - loss(logits - e)) / (2 * step)
        assert abs(difference.item() - d_logits[t, j].item()) <= step ** 2 * size[t].item() * 10 + 1e-9
