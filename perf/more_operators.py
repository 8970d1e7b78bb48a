"""Performance cases of the microscaled 4-bit operators and of layers of experts.

Rows are quantised to 4-bit floats with one power of two per 32 inputs, linear
layers multiply such rows by such weights, and in layers of experts each token
goes through the few it has chosen: the (token, choice) pairs are sorted by
expert, the rows gathered, multiplied expert by expert, and combined with the
token's weights.  Each case is one pass through one operator, either in plain
form (elementary torch operations in 32 bits, rounded once at the end) or,
with ``own`` set, through this package's entry points.

Formats and formulas, common to both forms:

- a block of 32 values x (the last of a row may be short) has the scale 2^e,
  e = max(floor(log2(max |x|)) - 2, -127), held as the byte e + 127, and the
  codes of x / 2^e: sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6, to the nearest (ties to
  the even code, more than 6 to 6); element 2 i is the low half of byte i;
- linear layers: y = bias + Q(x) W^T, Q as above, W in the same format;
- pairs: pair t * k + j is choice j of token t.  ``order`` lists them by expert,
  those of an expert in their order; ``position`` is the inverse; ``offsets``
  where each expert starts.  Pairs whose id is no expert's are dropped: -1 in
  ``position``, their places at the end of ``order`` are -1 and of gathered rows 0.
"""

import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the activations of one decoding step of 32 requests: latency
        dict(name="quantise_step", op="quantise", rows=32, cols=4096, dtype="bf16"),
        # a long prompt's activations: bytes
        dict(name="quantise_prompt", op="quantise", rows=8193, cols=8192, dtype="bf16"),
        # one token through the 7x7x512 -> 4096 fully connected shape of the benchmark: weights streamed once
        dict(name="linear_row", op="linear", rows=1, n_in=25088, n_out=4096, bias=False, dtype="bf16"),
        # a small batch of tokens through a layer of odd sizes, in full precision, with a bias
        dict(name="linear_rows_odd", op="linear", rows=13, n_in=5000, n_out=11003, bias=True, dtype="f32"),
        # the benchmark's batch of 256 through the fully connected shape: a product with few rows
        dict(name="linear_batch", op="linear", rows=256, n_in=25088, n_out=4096, bias=False, dtype="f16"),
        # a long prompt through a wide projection: a large matrix product
        dict(name="linear_prompt", op="linear", rows=8192, n_in=8192, n_out=8192, bias=False, dtype="bf16"),
        # one decoding step of 32 requests: a few rows for most experts, their weights streamed once
        dict(name="experts_step", op="experts", tokens=32, choices=4, experts=64, n_in=2048, n_out=2816, bias=False,
             dtype="bf16"),
        # a prompt of odd length: ragged matrix products, with a bias for each expert
        dict(name="experts_prompt", op="experts", tokens=4099, choices=4, experts=64, n_in=2048, n_out=2816, bias=True,
             dtype="bf16"),
        # the pairs of one decoding step among many experts, sorted, and their rows gathered: latency
        dict(name="dispatch_step", op="dispatch", tokens=32, choices=8, experts=256, width=4096, ids="i64", dtype="bf16"),
        # the pairs of a long prompt, some of them dropped, and their rows: bytes
        dict(name="dispatch_prompt", op="dispatch", tokens=8193, choices=4, experts=64, width=4096, ids="i32",
             dtype="bf16"),
        # the experts' results of a long prompt, weighted and added: bytes
        dict(name="combine_prompt", op="combine", tokens=8193, choices=4, experts=64, width=4096, dtype="f16"),
        # the gradients of both in full precision, rows of odd width: of the experts' results, the weights, the tokens
        dict(name="combine_gradient", op="gradient", tokens=2049, choices=6, experts=32, width=5003, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "linear", "linear", "experts", "experts", "dispatch", "combine", "gradient"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    size = _BYTES[dtype]
    if op == "quantise":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 9000), cols=_log(rng, 32, 12000), dtype=dtype)
            if rng.random() < 0.5:
                c["cols"] = max(64, c["cols"] // 64 * 64)
            if c["rows"] * c["cols"] * size <= 8193 * 8192 * 2:
                return c
    if op == "linear":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 9000), n_in=_log(rng, 200, 26000), n_out=_log(rng, 200, 12000),
                     bias=rng.random() < 0.5, dtype=dtype)
            if rng.random() < 0.5:
                c["n_in"], c["n_out"] = max(256, c["n_in"] // 128 * 128), max(256, c["n_out"] // 128 * 128)
            if c["rows"] * c["n_in"] * c["n_out"] <= 8192 ** 3 and c["n_in"] * c["n_out"] <= 25088 * 4096:
                return c
    if op == "experts":
        while True:
            c = dict(op=op, tokens=_log(rng, 1, 4100), choices=rng.choice([1, 2, 4, 6, 8]),
                     experts=rng.choice([8, 13, 32, 64, 128]), n_in=_log(rng, 200, 5000), n_out=_log(rng, 200, 5000),
                     bias=rng.random() < 0.5, dtype=dtype)
            if rng.random() < 0.5:
                c["n_in"], c["n_out"] = max(256, c["n_in"] // 128 * 128), max(256, c["n_out"] // 128 * 128)
            if (c["experts"] * c["n_in"] * c["n_out"] <= 64 * 2048 * 2816
                    and c["tokens"] * c["choices"] * c["n_in"] * c["n_out"] <= 4099 * 4 * 2048 * 2816):
                return c
    while True:
        c = dict(op=op, tokens=_log(rng, 1, 9000), choices=rng.choice([1, 2, 4, 6, 8]),
                 experts=rng.choice([8, 13, 32, 64, 128, 256]), width=_log(rng, 64, 8200), dtype=dtype)
        if rng.random() < 0.5:
            c["width"] = max(64, c["width"] // 64 * 64)
        if op == "dispatch":
            c["ids"] = rng.choice(["i32", "i64"])
        if c["tokens"] * c["choices"] * c["width"] * size <= (2049 * 6 * 5003 * 4 if op == "gradient"
                                                               else 8193 * 4 * 4096 * 2):
            return c


def work(case):
    op, size = case["op"], _BYTES[case["dtype"]]
    packed = lambda rows, cols: rows * (-(-cols // 2) + -(-cols // 32))  # noqa: E731
    if op == "quantise":  # read; write codes, scales and the values they stand for
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * size * n + packed(case["rows"], case["cols"]), "flops": 3 * n}
    if op == "linear":
        m, k, n = case["rows"], case["n_in"], case["n_out"]
        return {"bytes": packed(n, k) + size * m * (k + n) + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    pairs = case["tokens"] * case["choices"]
    if op == "experts":
        k, n = case["n_in"], case["n_out"]
        # weights of the experts that a token chooses, taken as independent choices of the uniform part
        used = case["experts"] * (1 - (1 - 1 / case["experts"]) ** pairs)
        return {"bytes": int(used * (packed(n, k) + (4 * n if case["bias"] else 0))) + size * (case["tokens"] * k + pairs * n)
                + 4 * pairs + 4 * case["experts"], "flops": 2 * pairs * n * k}
    d = case["width"]
    if op == "dispatch":
        return {"bytes": pairs * (8 + (8 if case["ids"] == "i64" else 4)) + 4 * case["experts"]
                + size * d * (case["tokens"] + pairs), "flops": pairs}
    if op == "combine":
        return {"bytes": 8 * pairs + size * d * (case["tokens"] + pairs), "flops": 2 * pairs * d}
    # dy, rows, weights -> d_rows, d_weights; gradient of the gathered rows -> dx
    return {"bytes": 12 * pairs + size * d * (3 * pairs + 2 * case["tokens"]), "flops": 4 * pairs * d}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, rows, cols, dtype):
    """Normal values, a few channels much larger than the rest."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= 1 + 7 * (torch.rand((cols,), generator=g, device="cuda") < 0.01)
    return x.to(dtype)


def _weights(g, rows, cols):
    """Codes and scales of a normal matrix: code bytes [rows, ceil(cols / 2)],
    scale bytes [rows, ceil(cols / 32)]; unused halves are 0."""
    magnitude = torch.tensor([0, 1, 1, 2, 2, 2, 3, 3, 3, 4, 4, 5, 5, 6, 6, 7], dtype=torch.uint8, device="cuda")
    r = torch.randint(0, 256, (rows, -(-cols // 2)), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(0, 4, r.shape, generator=g, device="cuda", dtype=torch.uint8)
    low = magnitude[(r & 15).int()] | ((s & 1) << 3)
    high = magnitude[(r >> 4).int()] | ((s >> 1) << 3)
    if cols % 2:
        high[:, -1] = 0
    scales = torch.randint(118, 121, (rows, -(-cols // 32)), generator=g, device="cuda", dtype=torch.uint8)
    return low | (high << 4), scales


def _ids(g, case):
    """Different experts for the choices of a token, some of them chosen more
    often than others; one pair in 50 dropped where there are many."""
    t, k, e = case["tokens"], min(case["choices"], case["experts"]), case["experts"]
    score = torch.randn((t, e), generator=g, device="cuda") + 0.5 * torch.randn((e,), generator=g, device="cuda")
    ids = torch.topk(score, k, dim=1).indices
    if t > 100:
        ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < 0.02, -1, ids)
    return ids.to(torch.int64 if case.get("ids") == "i64" else torch.int32)


def _linear_inputs(case, seed):
    g = _gen(seed)
    codes, scales = _weights(g, case["n_out"], case["n_in"])
    bias = torch.randn((case["n_out"],), generator=g, device="cuda") if case["bias"] else None
    return codes, scales, bias, _activations(g, case["rows"], case["n_in"], _DTYPES[case["dtype"]])


def _experts_inputs(case, seed):
    g = _gen(seed)
    e, n = case["experts"], case["n_out"]
    codes, scales = _weights(g, e * n, case["n_in"])
    bias = torch.randn((e, n), generator=g, device="cuda") if case["bias"] else None
    x = _activations(g, case["tokens"], case["n_in"], _DTYPES[case["dtype"]])
    return codes.view(e, n, -1), scales.view(e, n, -1), bias, x, _ids(g, case)


def _rows_inputs(case, seed):
    """ids, tokens' rows, the experts' result rows, weights that add up to 1,
    and two gradients."""
    g = _gen(seed)
    dtype = _DTYPES[case["dtype"]]
    ids = _ids(g, case)
    make = lambda rows: torch.randn((rows, case["width"]), generator=g, device="cuda").to(dtype)  # noqa: E731
    tokens, pairs = ids.shape[0], ids.numel()
    if case["op"] == "dispatch":
        return ids, make(tokens)
    weights = torch.softmax(torch.randn(ids.shape, generator=g, device="cuda"), 1)
    if case["op"] == "combine":
        return ids, make(pairs), weights
    return ids, make(pairs), weights, make(tokens), make(pairs)


# -------------------------------------------------------------- plain forms

def _plain_quantise(x):
    """What the quantised rows stand for, in fp32, with their codes and scale
    bytes."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -cols % 32)).view(rows, -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    byte = ((top.view(torch.int32) >> 23) - 2).clamp_(min=0)      # exponent field of the largest, less 2
    down = ((254 - byte) << 23).view(torch.float32)                # 2^-e, a normal number
    up = torch.where(byte > 0, byte << 23, 1 << 22).to(torch.int32).view(torch.float32)  # 2^e, 2^-127 for 0
    q = b * down
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp_(max=6.0)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code |= torch.signbit(q).to(torch.uint8) << 3
    values = (torch.copysign(a, q) * up).view(rows, -1)[:, :cols]
    return values, code[..., 0::2] | (code[..., 1::2] << 4), byte.to(torch.uint8)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _plain_dense(codes, scales, cols):
    """fp32 matrix of packed codes and scale bytes (of normal scales)."""
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    up = (scales.to(torch.int32) << 23).view(torch.float32)
    return table[c][..., :cols] * up.repeat_interleave(32, -1)[..., :cols]


def _plain_linear(s):
    x = s["x"]
    y = _plain_quantise(x)[0] @ _plain_dense(s["codes"], s["scales"], x.shape[1]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(x.dtype)


def _plain_order(ids, experts):
    flat = ids.reshape(-1).long()
    real = (flat >= 0) & (flat < experts)
    key = torch.where(real, flat, experts)
    order = torch.argsort(key, stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(flat.numel(), device=ids.device)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cumsum(counts, 0) - counts
    order = torch.where(real[order], order, -1)
    position = torch.where(real, position, -1).view(ids.shape)
    return offsets.to(torch.int32), order.to(torch.int32), position.to(torch.int32)


def _plain_gather(x, order, choices):
    rows = x[(order // choices).clamp_(min=0).long()]
    return torch.where((order >= 0)[:, None], rows, 0)


def _plain_experts(s):
    x, offsets, order = s["x"], s["offsets"], s["order"]
    q = _plain_gather(_plain_quantise(x)[0], order, s["choices"])
    y = torch.zeros((order.shape[0], s["codes"].shape[1]), device=x.device)
    bounds = offsets.tolist()  # the sizes of the experts' products
    for e in range(len(bounds) - 1):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        part = q[lo:hi] @ _plain_dense(s["codes"][e], s["scales"][e], x.shape[1]).t()
        y[lo:hi] = part if s["bias"] is None else part + s["bias"][e]
    return y.to(x.dtype)


def _plain_dispatch(s):
    offsets, order, position = _plain_order(s["ids"], s["experts"])
    return {"offsets": offsets, "order": order, "position": position,
            "rows": _plain_gather(s["x"], order, s["ids"].shape[1])}


def _taken(rows, position):
    """[tokens, choices, width] in fp32 of the rows of each token's pairs, 0 for dropped ones."""
    return torch.where((position >= 0)[..., None], rows[position.clamp(min=0).long()].float(), 0.0)


def _plain_combine(s):
    return (_taken(s["rows"], s["position"]) * s["weights"][..., None]).sum(1).to(s["rows"].dtype)


def _plain_gradient(s):
    dy, position, weights = s["dy"].float(), s["position"], s["weights"]
    taken = _taken(s["rows"], position)
    d_weights = (taken * dy[:, None]).sum(-1)
    d_rows = torch.zeros((position.numel() + 1, dy.shape[1]), device=dy.device)
    to = torch.where(position >= 0, position, position.numel()).long()  # the last row takes what is dropped
    d_rows[to.view(-1)] = (weights[..., None] * dy[:, None]).view(-1, dy.shape[1])
    return {"d_rows": d_rows[:-1].to(s["dy"].dtype), "d_weights": d_weights,
            "dx": _taken(s["d_gathered"], position).sum(1).to(s["dy"].dtype)}


# ------------------------------------------------------------- prepare and run

def prepare(case, seed):
    op = case["op"]
    s = {"op": op}
    if own:
        import popcount_convolution_amd as pca
    if op == "quantise":
        s["x"] = _activations(_gen(seed), case["rows"], case["cols"], _DTYPES[case["dtype"]])
    elif op == "linear":
        codes, scales, bias, s["x"] = _linear_inputs(case, seed)
        if own:
            s["layer"] = pca.MX4Linear(in_features=case["n_in"], out_features=case["n_out"], codes=codes, scales=scales,
                                       bias=bias)
        else:
            s.update(codes=codes, scales=scales, bias=bias)
    elif op == "experts":
        codes, scales, bias, s["x"], ids = _experts_inputs(case, seed)
        if own:
            s["layer"] = pca.MX4Experts(experts=case["experts"], in_features=case["n_in"], out_features=case["n_out"],
                                        codes=codes, scales=scales, bias=bias)
            s["order"] = pca.sort_by_expert(ids, case["experts"])
        else:
            offsets, order, _ = _plain_order(ids, case["experts"])
            s.update(codes=codes, scales=scales, bias=bias, offsets=offsets, order=order, choices=ids.shape[1])
    elif op == "dispatch":
        s["ids"], s["x"] = _rows_inputs(case, seed)
        s["experts"] = case["experts"]
    else:
        ids, s["rows"], s["weights"], *rest = _rows_inputs(case, seed)
        if op == "gradient":
            s["dy"], s["d_gathered"] = rest
        if own:
            s["order"] = pca.sort_by_expert(ids, case["experts"])
        else:
            s["position"] = _plain_order(ids, case["experts"])[2]
    return s


def run(state):
    s = state
    op = s["op"]
    if not own:
        if op == "quantise":
            return _plain_quantise(s["x"])[0].to(s["x"].dtype)
        return {"linear": _plain_linear, "experts": _plain_experts, "dispatch": _plain_dispatch,
                "combine": _plain_combine, "gradient": _plain_gradient}[op](s)
    import popcount_convolution_amd as pca
    if op == "quantise":
        _, values = pca.mx4_quantize(s["x"], values=True)
        return values
    if op == "linear":
        return s["layer"].forward(s["x"])
    if op == "experts":
        return s["layer"].forward(s["x"], s["order"])
    if op == "dispatch":
        order = pca.sort_by_expert(s["ids"], s["experts"])
        return {"offsets": order.offsets, "order": order.order, "position": order.position,
                "rows": order.gather(s["x"])}
    if op == "combine":
        return s["order"].combine(s["rows"], s["weights"])
    d_rows, d_weights = s["order"].combine_backward(s["dy"], s["rows"], s["weights"])
    return {"d_rows": d_rows, "d_weights": d_weights, "dx": s["order"].gather_backward(s["d_gathered"])}


# ----------------------------------------------- the definition, in 64 bits

def _exact_quantise(x):
    """Counts the midpoints between neighbouring magnitudes that a value has
    passed; one that it sits on counts where the code above is even."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[1], 32):
        b = x[:, at:at + 32].double()
        _, exponent = torch.frexp(b.abs().amax(1, keepdim=True))   # the largest is in [2^(exponent - 1), 2^exponent)
        e = torch.where(b.abs().amax(1, keepdim=True) > 0, exponent - 3, -127).clamp(min=-127)
        a = torch.ldexp(b.abs(), -e)
        index = torch.zeros_like(a, dtype=torch.int64)
        for i in range(7):
            middle = (_E2M1[i] + _E2M1[i + 1]) / 2
            index += (a >= middle) if i % 2 else (a > middle)
        value = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)[index]
        out[:, at:at + 32] = torch.ldexp(torch.where(b < 0, -value, value), e)
    return out


def _exact_matrix(codes, scales, cols):
    """A code s m1 m2 m3 is (-1)^s times m3 / 2 where m1 m2 = 0, otherwise
    (1 + m3 / 2) 2^(m1m2 - 1)."""
    out = torch.empty((codes.shape[0], cols), dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = ((codes >> 4) if half else (codes & 15)).int()
        exponent, fraction = (c >> 1) & 3, (c & 1).double() / 2
        v = torch.where(exponent == 0, fraction, torch.ldexp(1 + fraction, exponent - 1))
        block = scales.repeat_interleave(16, 1)[:, :c.shape[1]].int() - 127
        v = torch.ldexp(torch.where(c >= 8, -v, v), block)
        width = out[:, half::2].shape[1]
        out[:, half::2] = v[:, :width]
    return out


def _exact_experts(case, seed):
    codes, scales, bias, x, ids = _experts_inputs(case, seed)
    q = _exact_quantise(x)
    y = torch.zeros((ids.numel(), case["n_out"]), dtype=torch.float64, device="cuda")
    at = 0
    for e in range(case["experts"]):
        token = torch.nonzero(ids == e)[:, 0]  # by token, then by choice
        n = token.shape[0]
        if n:
            w = _exact_matrix(codes[e], scales[e], case["n_in"])
            y[at:at + n] = torch.matmul(q[token], w.t().contiguous())
            if bias is not None:
                y[at:at + n] += bias[e].double()
        at += n
    return y


def _exact_positions(ids, experts):
    """Place of each pair, counted pair by pair of one expert after the other; -1 where dropped."""
    position = torch.full(ids.shape, -1, dtype=torch.int64, device=ids.device)
    at = 0
    for e in range(experts):
        chosen = ids == e
        n = int(chosen.sum())
        position[chosen] = at + torch.arange(n, device=ids.device)
        at += n
    return position


def exact(case, seed):
    op = case["op"]
    if op == "quantise":
        return _exact_quantise(_activations(_gen(seed), case["rows"], case["cols"], _DTYPES[case["dtype"]]))
    if op == "linear":
        codes, scales, bias, x = _linear_inputs(case, seed)
        w = _exact_matrix(codes, scales, case["n_in"])
        y = torch.matmul(_exact_quantise(x), w.t().contiguous())
        return y if bias is None else y + bias.double()
    if op == "experts":
        return _exact_experts(case, seed)
    ids, *rest = _rows_inputs(case, seed)
    position = _exact_positions(ids, case["experts"])
    pairs, choices = ids.numel(), ids.shape[1]
    where = position.view(-1)
    kept = torch.nonzero(where >= 0)[:, 0]
    if op == "dispatch":
        rows = torch.zeros((pairs, case["width"]), dtype=torch.float64, device="cuda")
        rows[where[kept]] = rest[0].double()[kept // choices]
        return {"offsets": None, "order": None, "position": None, "rows": rows}
    tokens, width = ids.shape[0], case["width"]

    def back(rows, weights):
        out = torch.zeros((tokens, width), dtype=torch.float64, device="cuda")
        for j in range(choices):  # one choice of every token at a time
            have = torch.nonzero(position[:, j] >= 0)[:, 0]
            part = rows[position[have, j]].double()
            out[have] += part if weights is None else part * weights[have, j].double()[:, None]
        return out

    if op == "combine":
        return back(rest[0], rest[1])
    rows, weights, dy, d_gathered = rest
    d_rows = torch.zeros((pairs, width), dtype=torch.float64, device="cuda")
    d_weights = torch.zeros((tokens, choices), dtype=torch.float64, device="cuda")
    for j in range(choices):
        have = torch.nonzero(position[:, j] >= 0)[:, 0]
        grad = dy[have].double()
        d_rows[position[have, j]] = grad * weights[have, j].double()[:, None]
        d_weights[have, j] = (grad * rows[position[have, j]].double()).sum(1)
    return {"d_rows": d_rows, "d_weights": d_weights, "dx": back(d_gathered, None)}
