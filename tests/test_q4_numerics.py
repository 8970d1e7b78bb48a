"""How exact the 4-bit operators are, at the ends of their types' ranges and in
ordinary use, against 64-bit references."""

import numpy as np
import pytest
import torch

import popcount_convolution_amd as pca
import q4_precision as prec
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


# ------------------------------------------- more than one launch can take

@pytest.mark.gpu
@pytest.mark.parametrize("k,n,dtype", [(40, 5, "bf16"), (300, 20, "f32"), (300, 40, "f16")])
def test_linear_more_rows_than_a_launch(dev, k, n, dtype):
    """2^18 rows and some: every row is computed, rows of the last launch like
    the same rows of the first."""
    print("linear rows", k, n, dtype, flush=True)
    rng = np.random.default_rng(k + n)
    rows, tail = (1 << 18) + 1037, 1037
    codes = rng.integers(0, 16, (n, k))
    scales = (rng.uniform(0.3, 1.5, (n, -(-k // 64))) * 0.02).astype(np.float16)
    words = pca.pack_codes(codes)
    layer = pca.Q4Linear(in_features=k, out_features=n, weight_words=words, scales=scales, group=64)
    x = torch.randn(rows, k, device=dev).to(DT[dtype])
    x[-tail:] = x[:tail]
    buf = torch.full((rows, n + 1), 7.0, device=dev, dtype=DT[dtype])
    y = layer.forward(x, out=buf[:, :n])
    assert torch.equal(y[-tail:], y[:tail]) and bool((buf[:, n] == 7.0).all())
    some = torch.cat([torch.arange(0, rows, 997), torch.arange((1 << 18) - 50, (1 << 18) + 50)]).to(dev)
    want, mass = ref.linear(host(x[some]), words, scales, None, None, 64)
    assert (np.abs(host(y[some]) - want) <= ref.linear_bound(want, mass, None, k, 64, dtype)).all()
    assert layer.workspace_bytes(2 ** 31 - 1, DT[dtype]) == layer.workspace_bytes(1 << 20, DT[dtype])


@pytest.mark.gpu
def test_attention_more_workgroups_than_a_launch(dev):
    """2^24 workgroups: 256 requests, one with 32768 - 255 queries and the others
    with one, and no max_q.  The same as with each request's own."""
    print("attention workgroups", flush=True)
    requests, total, heads, kv, dim, block = 256, 32768, 32, 8, 64, 16
    lens = torch.full((requests,), 40, dtype=torch.int32, device=dev)
    lens[200] = total
    counts = torch.ones(requests, dtype=torch.int64, device=dev)
    counts[200] = total - 255
    starts = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)).to(torch.int32)
    width = total // block
    cache = pca.KV4Cache(width, block, kv, dim)
    x = torch.randn(width * block, kv, dim, device=dev)
    cache.append(x, x, torch.arange(width * block, dtype=torch.int32, device=dev))
    table = torch.arange(width, dtype=torch.int32, device=dev).repeat(requests, 1)
    q = torch.randn(total, heads, dim, device=dev).bfloat16()
    out = cache.attention(q, table, lens, q_start=starts, window=50)
    for r in (0, 1, 199, 200, 201, 255):
        a, b = int(starts[r]), int(starts[r + 1])
        one = cache.attention(q[a:b], table[r:r + 1], lens[r:r + 1], window=50)
        assert float((out[a:b] - one).float().abs().max()) <= 2.0 ** -6, r


@pytest.mark.gpu
def test_attention_more_columns_than_a_join(dev):
    """2^23 columns whose two parts are joined, of which 100 have a query."""
    print("attention columns", flush=True)
    requests, kv, heads, dim, block, width = 16384, 8, 64, 64, 16, 600
    cache = pca.KV4Cache(width, block, kv, dim)
    x = torch.randn(width * block, kv, dim, device=dev)
    cache.append(x, x, torch.arange(width * block, dtype=torch.int32, device=dev))
    table = torch.arange(width, dtype=torch.int32, device=dev).repeat(requests, 1)
    owner = torch.arange(0, requests, 164, device=dev)[:100]
    owner[-1] = requests - 1
    counts = torch.zeros(requests, dtype=torch.int64, device=dev)
    counts[owner] = 1
    starts = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)).to(torch.int32)
    lens = torch.full((requests,), width * block, dtype=torch.int32, device=dev)
    q = torch.randn(100, heads, dim, device=dev).bfloat16()
    out = cache.attention(q, table, lens, q_start=starts, max_q=8)
    want = cache.attention(q, table[:100], lens[:100])
    assert float((out - want).float().abs().max()) <= 2.0 ** -6


@pytest.mark.gpu
def test_append_more_rows_than_a_launch(dev):
    """2^27 rows of 256 channels and some (2^24 tokens of 8 heads, one row
    expanded): the last tokens are written."""
    print("append rows", flush=True)
    tokens = (1 << 24) + 5
    k = torch.randn(1, 1, 256, device=dev).bfloat16().expand(tokens, 8, 256)
    cache, small = pca.KV4Cache(2, 16, 8, 256), pca.KV4Cache(2, 16, 8, 256)
    slots = torch.full((tokens,), -1, dtype=torch.int32, device=dev)
    slots[-20:] = torch.arange(20, dtype=torch.int32, device=dev)
    cache.append(k, k, slots)
    small.append(k[:20], k[:20], torch.arange(20, dtype=torch.int32, device=dev))
    assert torch.equal(cache.pool, small.pool)


# ----------------------------------------------------------- small fp32 rows

@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("rows,n", [(5, 90), (70, 300), (20, 9000), (50, 9000), (70, 9000)])
def test_linear_fp32_small_rows(dev, rows, n, group, zeros):
    """fp32 rows of 1e-26 to 1e-35 times scales of 1e-4, at every batch size: as
    exact as rows of any other size, as long as the results are normal numbers.
    2000 terms of random signs: their split to 2^-23 and one fp32 rounding for each
    of at most 16 + 63 partial sums a result (a matrix instruction adds 16 or 32
    terms, then groups and splits are added) are below 2^-20 of the results' rms."""
    print("small rows", rows, n, group, zeros, flush=True)
    rng = np.random.default_rng(rows + n + group)
    k = 2000
    codes = rng.integers(0, 16, (n, k))
    scales = (rng.uniform(0.5, 1.5, (n, -(-k // group))) * 1e-4).astype(np.float16)
    zs = rng.integers(6, 10, scales.shape).astype(np.uint8) if zeros else None
    words = pca.pack_codes(codes)
    layer = pca.Q4Linear(in_features=k, out_features=n, weight_words=words, scales=scales, zeros=zs, group=group)
    x = (rng.normal(0, 1, (rows, k)) * 10.0 ** np.linspace(-35, -26, rows)[:, None]).astype(np.float32)
    want, _ = ref.linear(x.astype(np.float64), words, scales, zs, None, group)
    err = host(layer.forward(torch.from_numpy(x).to(dev))) - want
    rms = lambda a: np.sqrt((a ** 2).mean(1))  # noqa: E731
    assert rms(want).min() > 2.0 ** -126
    ratio = rms(err) / rms(want)
    assert (ratio <= 2.0 ** -20).all(), ratio.max()


# -------------------------------------------------------- ordinary precision

LINEAR = [  # one row and few (1 to 4 output tiles a workgroup, 8 or 16 waves), many (32, 64, 128 rows), split and whole
    (1, 32, 16, 32, False, False),
    (1, 4096, 96, 128, False, False),
    (1, 8200, 8100, 64, True, True),
    (3, 127, 33, 128, False, True),
    (7, 2500, 5000, 32, False, False),
    (13, 5000, 11003, 64, True, True),
    (16, 256, 16000, 64, True, False),
    (17, 8200, 4100, 64, True, True),
    (50, 4100, 4111, 128, True, False),
    (130, 2049, 3500, 32, True, True),
    (300, 1100, 3100, 128, False, False),
    (2000, 300, 1400, 32, False, True),
]


def linear_case(rows, k, n, group, zeros, bias):
    rng = np.random.default_rng(rows * 1009 + k + n)
    codes = rng.integers(0, 16, (n, k))
    shape = (n, -(-k // group))
    scales = (rng.uniform(0.3, 1.5, shape) * 0.02).astype(np.float16)
    zs = rng.integers(5, 11, shape).astype(np.uint8) if zeros else None
    b = rng.normal(0, 1, n).astype(np.float32) if bias else None
    return pca.pack_codes(codes), scales, zs, b, rng.normal(0, 1, (rows, k)).astype(np.float32)


@pytest.mark.parametrize("case", LINEAR[1:4] + LINEAR[-1:])
def test_linear_bound_tells_one_part_from_two(case):
    """The bound that the kernels are held to passes two fp16 parts of x and
    fails one."""
    *w, x = linear_case(*case)
    want, bound = prec.linear(x, *w, case[3])
    for count in (1, 2):
        top = np.abs(x).max(1, keepdims=True)
        got = prec.linear(prec.parts(x, count, top), *w, case[3])[0]
        assert (prec.rms((got - want) / bound) <= 1) == (count == 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", LINEAR)
def test_linear_precision(dev, dtype, case):
    """fp32: the rms error is that of two-part operands and fp32 sums.  16-bit
    types: that of one rounding of the result, and 5% (fp32 sums with the codes'
    offset in them, at most a tenth of fp16's rounding)."""
    print("linear precision", dtype, case, flush=True)
    words, scales, zs, b, x = linear_case(*case)
    rows, k, n, group, *_ = case
    layer = pca.Q4Linear(in_features=k, out_features=n, weight_words=words, scales=scales, zeros=zs, bias=b,
                         group=group)
    x = torch.from_numpy(x).to(dev).to(DT[dtype])
    want, bound = prec.linear(host(x), words, scales, zs, b, group)
    err = host(layer.forward(x)) - want
    if dtype == "f32":
        ratio = prec.rms(err / bound)
        assert ratio <= 1, ratio
    else:
        best = host(torch.from_numpy(want).to(DT[dtype])) - want
        assert prec.rms(err) <= 1.05 * prec.rms(best), (prec.rms(err), prec.rms(best))


def attention_case(lens, kv, dim, group, seed):
    """Keys, values and steps of each request in 64 bits, as the cache holds them."""
    rng = np.random.default_rng(seed)
    k = [rng.normal(0, 1, (n, kv, dim)).astype(np.float32) for n in lens]
    v = [rng.normal(0, 1, (n, kv, dim)).astype(np.float32) for n in lens]
    kx = [ref.quantise(a, group)[3].astype(np.float64) for a in k]
    vq = [ref.quantise(a, group) for a in v]
    return rng, k, v, kx, [a[3].astype(np.float64) for a in vq], [a[1].astype(np.float64).max(-1) for a in vq]


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("length", [45, 703])
def test_attention_bound_tells_one_part_from_two(dim, group, length):
    """The bound fails queries in one fp16 part, probabilities times steps in one, and
    passes both in two."""
    rng, _, _, kx, vx, step = attention_case([length], 1, dim, group, dim + length)
    q = rng.normal(0, 1.5, (1, 4, dim))
    want, _, bound, _ = prec.attention(q, kx, vx, step, [length], [1], dim ** -0.5, group)
    z = np.einsum("hd,td->ht", q[0], kx[0][:, 0]) * dim ** -0.5
    for count in (1, 2):
        split = prec.parts(q, count, np.abs(q).max(-1, keepdims=True))
        got = prec.attention(split, kx, vx, step, [length], [1], dim ** -0.5, group)[0]
        assert (prec.rms((got - want) / bound) <= 1) == (count == 2)
        p = np.exp(z - z.max(1, keepdims=True))
        got = prec.parts(p, count, 1.0) / p.sum(1, keepdims=True) @ vx[0][:, 0]
        assert (prec.rms((got - want[0]) / bound[0]) <= 1) == (count == 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,group", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 128), (256, 64),
                                       (256, 32), (120, 64), (80, 32), (136, 64)])
@pytest.mark.parametrize("ratio,lens,counts", [(1, [703, 45], [1, 1]), (8, [703, 45], [1, 1]), (4, [6000], [1]),
                                               (16, [6000], [1]), (2, [300, 37], [20, 37])])
def test_attention_precision(dev, dtype, dim, group, ratio, lens, counts):
    """fp32: the rms errors of the result and the log-sum-exp are those of two-part
    operands and fp32 sums.  fp16: that of one rounding of the result, and 10%
    (probabilities to 2^-16, a 32nd of it).  bf16: and a quarter (probabilities to
    2^-11, an eighth of it, in terms of up to a few times the result)."""
    print("attention precision", dtype, dim, group, ratio, lens, counts, flush=True)
    kv, block = 2, 16
    rng, k, v, kx, vx, step = attention_case(lens, kv, dim, group, dim * 31 + group + ratio + sum(lens))
    per = [-(-n // block) for n in lens]
    cache = pca.KV4Cache(sum(per), block, kv, dim, group=group)
    order = rng.permutation(sum(per)).astype(np.int32)
    table = np.full((len(lens), max(per)), -1, np.int32)
    for r, n in enumerate(per):
        table[r, :n] = order[sum(per[:r]):sum(per[:r + 1])]
        pos = np.arange(lens[r])
        up = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
        cache.append(up(k[r]), up(v[r]), up((table[r, pos // block] * block + pos % block).astype(np.int32)))
    q = torch.from_numpy(rng.normal(0, 1.5, (sum(counts), kv * ratio, dim)).astype(np.float32)).to(dev).to(DT[dtype])
    starts = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(dev)
    lse = torch.empty(q.shape[:2], device=dev)
    out = cache.attention(q, up(table), up(np.array(lens, np.int32)), q_start=starts, max_q=max(counts), lse=lse)
    want, want_lse, bound, lse_bound = prec.attention(host(q), kx, vx, step, lens, counts, dim ** -0.5, group)
    err = host(out) - want
    if dtype == "f32":
        assert prec.rms(err / bound) <= 1, prec.rms(err / bound)
        assert prec.rms((host(lse) - want_lse) / lse_bound) <= 1
    else:
        best = host(torch.from_numpy(want).to(DT[dtype])) - want
        assert prec.rms(err) <= {"f16": 1.1, "bf16": 1.25}[dtype] * prec.rms(best), (prec.rms(err), prec.rms(best))


# ------------------------------------------------- the ends of bf16's range

@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("rows,n", [(9, 90), (70, 300), (20, 9000), (50, 9000), (70, 9000)])
def test_linear_bf16_ends(dev, rows, n, group, zeros):
    """Finite bf16 rows up to the type's largest, of mixed signs and of one, and down
    to its subnormals: the results are finite, and off by one rounding of theirs and
    fp32 sums (or of bf16's smallest subnormal steps)."""
    print("bf16 ends", rows, n, group, zeros, flush=True)
    rng = np.random.default_rng(rows + n + group)
    k = 300
    codes = rng.integers(0, 16, (n, k))
    scales = (rng.uniform(0.5, 1.5, (n, -(-k // group))) * 1e-4).astype(np.float16)
    zs = rng.integers(0, 16, scales.shape).astype(np.uint8) if zeros else None
    words = pca.pack_codes(codes)
    layer = pca.Q4Linear(in_features=k, out_features=n, weight_words=words, scales=scales, zeros=zs, group=group)
    x = rng.uniform(0.5, 1, (rows, k)) * rng.choice([-1, 1], (rows, k))
    x[::3] = np.abs(x[::3])
    x *= 2.0 ** np.array([128, 127, 124, 118, 112, 0, -100, -112, -120])[np.arange(rows) % 9][:, None]
    x = torch.from_numpy(np.clip(x, -3.3e38, 3.3e38).astype(np.float32)).to(dev).bfloat16()
    assert bool(x.isfinite().all())
    want, bound = prec.linear(host(x), words, scales, zs, None, group)
    got = host(layer.forward(x))
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= ref.ROUND["bf16"] * np.abs(want) + 8 * bound + 2.0 ** -133).all()


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [2, 16])
@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32), (128, 128), (256, 128)])
def test_attention_bf16_query_ends(dev, dim, group, heads):
    """Queries of 2^-110 to bf16's largest with the scale that undoes it give the
    results of queries of ordinary size, to their roundings: powers of two change
    nothing else."""
    print("query ends", dim, group, heads, flush=True)
    n = 200
    rng = np.random.default_rng(dim + group + heads)
    cache = pca.KV4Cache(13, 16, 2, dim, group=group)
    k, v = (torch.from_numpy(rng.normal(0, 1, (n, 2, dim)).astype(np.float32)).to(dev) for _ in range(2))
    cache.append(k, v, torch.arange(n, dtype=torch.int32, device=dev))
    table = torch.arange(13, dtype=torch.int32, device=dev)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    q = torch.from_numpy(rng.uniform(-1, 1, (1, heads, dim))).to(dev).bfloat16()
    q[0, 0] = q[0, 0].abs()
    want = cache.attention(q, table, lens, scale=2.0)
    for e in (-110, -60, 60, 100, 110, 114, 118, 124, 127):
        big = (q.double() * 2.0 ** e).bfloat16()
        assert bool(big.isfinite().all())
        assert torch.equal(cache.attention(big, table, lens, scale=2.0 * 2.0 ** -e), want), e  # a normal number
