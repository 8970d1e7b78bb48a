"""How exact the 4-bit operators are, at the ends of their types' ranges and in
ordinary use, against 64-bit references."""

import numpy as np
import pytest
import torch

import popcount_convolution_amd as pca
import q4_reference as ref

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pca.load_library()
    return torch.device("cuda:0")


def host(t):
    return t.to(torch.float64).cpu().numpy()


# ---------------------------------------------------------- extreme logits

LN2 = 0.6931472  # as a float, times log2 e this is 1 in fp32: logits are in base 2


def test_base_two_scale():
    assert np.float32(LN2) * np.float32(1.4426950408889634) == 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64), (256, 128), (128, 32)])
@pytest.mark.parametrize("heads", [1, 8])
@pytest.mark.parametrize("length,first,second", [
    (1, 0, None),       # a lone token
    (300, 0, 256),      # the same wave's next tile
    (300, 256, 0),
    (300, 3, 4),        # one tile
    (300, 290, None),   # late, behind far lower ones
])
def test_attention_extreme_logits(dev, dtype, dim, group, heads, length, first, second):
    """Logits of 2^20 to 2^40 (fp16 queries: 2^30) of both signs, exact in fp32:
    token `first` has z, `second` one fp32 step more, the others -|z| or so, and
    values have steps of 3e-5 to 3.  The softmax is finite however coarse the
    logits are, and exact up to its own roundings: probabilities in 11, 16 or 23
    bits times codes of up to 8 steps, fp32 sums of up to 64 terms with the offset
    of the codes, exp2 to 2^-20, and the result's rounding."""
    print("extreme logits", dtype, dim, group, heads, length, first, second, flush=True)
    cases = [(e, sign, step) for e in range(20, 31 if dtype == "f16" else 41) for sign in (1, -1)
             for step in (3e-5, 2e-4, 1.9e-3, 0.1, 3.0)]
    n, block = len(cases), 16
    rng = np.random.default_rng(dim + group + heads + length)
    per = -(-length // block)
    cache = pca.KV4Cache(n * per, block, 1, dim, group=group)
    table = np.arange(n * per, dtype=np.int32).reshape(n, per)
    slots = np.concatenate([table[:, p // block, None] * block + p % block for p in range(length)], 1)
    lift = 15 if dtype == "f16" else 0  # a part of the logit that the keys bring
    k = np.zeros((n, length, 1, dim), np.float32)
    v = np.zeros_like(k)
    q = np.zeros((n, heads, dim), np.float32)
    z = np.zeros((n, length))
    for i, (e, sign, step) in enumerate(cases):
        a = 1.296875 * 2.0 ** lift
        k[i, :, 0, :group] = -sign * a
        k[i, first, 0, :group] = a
        if second is not None:
            k[i, second, 0, :group] = a
            k[i, second, 0, group:2 * group] = 1.0
        q[i, :, 0] = sign * 2.0 ** (e - lift)
        q[i, :, group] = 2.0 ** (e - 23)
        z[i] = k[i, :, 0, 0].astype(np.float64) * q[i, 0, 0] + k[i, :, 0, group].astype(np.float64) * q[i, 0, group]
        v[i] = rng.uniform(0, 15 * step, v[i].shape)
    up = lambda x: torch.from_numpy(x).to(dev)  # noqa: E731
    rows = lambda x: up(x.reshape(n * length, 1, dim))  # noqa: E731
    kv, vv = cache.append(rows(k), rows(v), up(slots.reshape(-1).astype(np.int32)), values=True)
    assert torch.equal(kv.cpu(), torch.from_numpy(k.reshape(n * length, 1, dim)))
    lse = torch.empty(n, heads, device=dev)
    out = cache.attention(up(q).to(DT[dtype]), up(table), torch.full((n,), length, dtype=torch.int32, device=dev),
                          scale=LN2, lse=lse)
    p = 2.0 ** (z - z.max(1, keepdims=True))
    want = np.einsum("il,ild->id", p / p.sum(1, keepdims=True), host(vv).reshape(n, length, dim))[:, None]
    step = np.array([c[2] for c in cases])[:, None, None]
    bits = {"bf16": 2.0 ** -11, "f16": 2.0 ** -16, "f32": 2.0 ** -23}[dtype]
    offset = {"bf16": 1039, "f16": 143, "f32": 8}[dtype]
    bound = (ref.ROUND[dtype] * (1 + 2.0 ** -7) * np.abs(want) + step * (8 * bits + ref.EPS * 64 * offset) +
             15 * step * 2.0 ** -20 + ref.TINY[dtype])
    bad = ~(np.abs(host(out) - want) <= bound)
    assert not bad.any(), [cases[i] for i in np.flatnonzero(bad.any((1, 2)))]
    top = (z.max(1) + np.log2(p.sum(1)))[:, None] * np.log(2)
    assert (np.abs(host(lse) - top) <= 2.0 ** -21 * np.abs(top)).all()


# ------------------------------------------------------------ long lengths

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [1, 8])
@pytest.mark.parametrize("window", [5090, 100, 0])
def test_attention_lengths_near_32_bits(dev, dtype, heads, window):
    """Lengths up to 2^31 - 1 over a table of 8000 tokens: a query whose window
    lies past the table sees nothing, in one part or eleven (whose last starts past
    2^31 where the first starts at the window), and the requests
    beside it are as they are alone."""
    print("lengths", dtype, heads, window, flush=True)
    rng = np.random.default_rng(window)
    lens = [7000, 2 ** 31 - 1, 2 ** 31 - 40, 2 ** 31 - 700, 2 ** 30, 8000 + 5000, 0]
    block, width, dim = 16, 500, 64
    cache = pca.KV4Cache(width, block, 1, dim, group=64)
    x = [torch.from_numpy(rng.normal(0, 1, (width * block, 1, dim)).astype(np.float32)).to(dev) for _ in range(2)]
    cache.append(*x, torch.arange(width * block, dtype=torch.int32, device=dev))
    table = torch.arange(width, dtype=torch.int32, device=dev).repeat(len(lens), 1)
    q = torch.from_numpy(rng.normal(0, 1, (len(lens), heads, dim)).astype(np.float32)).to(dev).to(DT[dtype])
    lse = torch.empty(len(lens), heads, device=dev)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    out = cache.attention(q, table, n, window=window, lse=lse)
    alone = cache.attention(q[:1], table[:1], n[:1], window=window)
    whole = cache.attention(q, table, n.clamp(max=width * block))  # without a window all of the table is seen
    bound = {"bf16": 2.0 ** -7, "f32": 2.0 ** -16}[dtype]  # parts end elsewhere; values are below 4
    assert float((out[:1] - alone).abs().max()) <= 4 * bound
    for r, length in enumerate(lens):
        if length == 0 or window and length - window >= width * block:
            assert not out[r].any() and bool(torch.isneginf(lse[r]).all())
        else:
            assert bool(out[r].any()) and bool(lse[r].isfinite().all())
            if not window:
                assert float((out[r] - whole[r]).abs().max()) <= 4 * bound
