"""Performance cases of the low-bit decoding operators.

A decoding step with everything in 4 bits: linear layers with 4-bit weights
and group scales, the write of new keys and values into a paged 4-bit cache,
attention over that cache, and the block tables and slot maps that say where
tokens go.  Each case is one pass through one operator, either in plain form
(elementary torch operations in 32 bits, rounded once at the end) or, with
``own`` set, through this package's entry points.

Formats, common to both forms:

- weights: 4-bit codes c, input i at bits 4 * (i % 8) of word i // 8, with an
  fp16 scale s per group of inputs and an optional zero point z (8 without):
  w = s * (c - z);
- cache rows: per token, head and group of channels an fp16 step s and an fp16
  midpoint b, x = s * (c - 8) + b, where s = fp16((max - min) * fp32(1/15)),
  b = fp16(min + 8 s), c = clamp(rint((x - b) * (1 / s)) + 8, 0, 15), each
  step rounded to fp32.
"""

import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token through a small projection: the latency of a call
        dict(name="linear_row_small", op="linear", rows=1, n_in=512, n_out=512, group=32, zeros=False, bias=False,
             dtype="bf16"),
        # one token through the 7x7x512 -> 4096 fully connected shape of the benchmark: weights streamed once
        dict(name="linear_row_wide", op="linear", rows=1, n_in=25088, n_out=4096, group=128, zeros=False, bias=False,
             dtype="bf16"),
        # a small batch of tokens through a layer of odd sizes, in full precision, with zero points and a bias
        dict(name="linear_rows_odd", op="linear", rows=13, n_in=5000, n_out=11003, group=64, zeros=True, bias=True,
             dtype="f32"),
        # the benchmark's batch of 256 through the same fully connected shape: a matrix product
        dict(name="linear_batch_wide", op="linear", rows=256, n_in=25088, n_out=4096, group=128, zeros=True,
             bias=False, dtype="bf16"),
        # a single user's next token early in a conversation: latency
        dict(name="attend_one", op="attend", requests=1, ctx=777, ragged=False, q_len=1, heads=8, kv_heads=2, dim=64,
             group=32, block=16, window=0, dtype="bf16"),
        # a serving batch: one token each over ragged contexts, grouped heads, one idle slot of length zero
        dict(name="attend_batch", op="attend", requests=32, ctx=8192, ragged=True, q_len=1, heads=32, kv_heads=8,
             dim=128, group=64, block=32, window=0, dtype="bf16"),
        # two users with very long contexts and a single shared key/value head: work split over the long axis
        dict(name="attend_long", op="attend", requests=2, ctx=131071, ragged=True, q_len=1, heads=16, kv_heads=1,
             dim=128, group=128, block=64, window=0, dtype="f16"),
        # prompts fed in chunks behind cached tokens, an odd head size, a sliding window, full precision
        dict(name="attend_prompt", op="attend", requests=3, ctx=4111, ragged=True, q_len=300, heads=10, kv_heads=5,
             dim=80, group=32, block=16, window=2000, dtype="f32"),
        # one new token for each of 32 requests: latency
        dict(name="append_step", op="append", tokens=32, kv_heads=8, dim=128, group=64, block=32, dtype="bf16"),
        # a long prompt's keys and values, views into a fused projection
        dict(name="append_prompt", op="append", tokens=8193, kv_heads=8, dim=128, group=64, block=16, dtype="bf16"),
        # the tables of one decoding step of 32 requests
        dict(name="tables_step", op="tables", requests=32, ctx=8192, new=1, block=32),
        # the tables of a large batch of ragged prompts, some behind cached tokens
        dict(name="tables_prompt", op="tables", requests=300, ctx=2000, new=600, block=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "attend", "attend", "append", "tables"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "linear":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 300), n_in=_log(rng, 200, 26000), n_out=_log(rng, 200, 12000),
                     group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, bias=rng.random() < 0.5, dtype=dtype)
            if rng.random() < 0.5:
                c["n_in"] = max(256, c["n_in"] // 128 * 128)
                c["n_out"] = max(256, c["n_out"] // 128 * 128)
            if 3072 in (c["n_in"], c["n_out"], c["rows"]):
                continue
            if c["rows"] * c["n_in"] * c["n_out"] <= 256 * 25088 * 4096 and c["n_in"] * c["n_out"] <= 25088 * 4096:
                return c
    if op == "attend":
        while True:
            kv = rng.choice([1, 2, 4, 5, 8])
            c = dict(op=op, requests=_log(rng, 1, 40), ctx=_log(rng, 40, 131071), ragged=rng.random() < 0.8,
                     q_len=1 if rng.random() < 0.6 else _log(rng, 2, 300), heads=kv * rng.choice([1, 2, 4, 7, 8]),
                     kv_heads=kv, dim=rng.choice([64, 80, 96, 128, 128, 256]), group=rng.choice([32, 64]),
                     block=rng.choice([16, 32, 64]), window=rng.choice([0, 0, 0, _log(rng, 16, 4000)]), dtype=dtype)
            if 3072 in (c["ctx"], c["window"]) or c["q_len"] > c["ctx"]:
                continue
            rows = c["requests"] * c["ctx"]
            if rows * kv * c["dim"] <= 32 * 8192 * 8 * 128 and rows * c["heads"] * c["q_len"] <= 1 << 26:
                return c
    if op == "append":
        while True:
            c = dict(op=op, tokens=_log(rng, 1, 8193), kv_heads=rng.choice([1, 2, 4, 5, 8]),
                     dim=rng.choice([64, 80, 96, 128, 128, 256]), group=rng.choice([32, 64]),
                     block=rng.choice([16, 32, 64]), dtype=dtype)
            if c["tokens"] != 3072 and c["tokens"] * c["kv_heads"] * c["dim"] * _BYTES[dtype] <= 8193 * 8 * 128 * 2:
                return c
    while True:
        c = dict(op=op, requests=_log(rng, 1, 512), ctx=_log(rng, 1, 8192), new=_log(rng, 1, 600),
                 block=rng.choice([16, 32, 64]))
        if 3072 not in (c["ctx"],) and c["requests"] * c["new"] <= 300 * 600:
            return c


# ------------------------------------------------ sizes that follow from a case

def _lengths(case):
    """Host lengths of an attention or tables case (a function of the case
    alone): cached-plus-new lengths and new tokens per request."""
    r = np.random.default_rng(1234 + case["requests"] * 7 + case["ctx"])
    n = case["requests"]
    if case["op"] == "attend":
        q = np.full(n, case["q_len"])
        ctx = np.full(n, case["ctx"])
        if case["ragged"]:
            ctx = r.integers(max(1, case["ctx"] // 4), case["ctx"] + 1, n)
            ctx[0] = case["ctx"]
            if case["q_len"] > 1:
                q = r.integers(1, case["q_len"] + 1, n)
                q[0] = case["q_len"]
            elif n > 2:
                ctx[n // 2] = 0  # an idle slot of the batch
            ctx = np.where(ctx > 0, np.maximum(ctx, q), 0)
        return ctx.astype(np.int64), q.astype(np.int64)
    new = np.full(n, 1) if case["new"] == 1 else r.integers(0, case["new"] + 1, n)
    ctx = r.integers(0, case["ctx"] + 1, n)
    if case["new"] > 1:
        ctx[::2] = 0  # fresh prompts
    return ctx.astype(np.int64), new.astype(np.int64)


def _visible(case):
    """(visible key positions summed over requests, query-key pairs summed)."""
    ctx, q = _lengths(case)
    w = case["window"]
    keys = pairs = 0
    for c, n in zip(ctx.tolist(), q.tolist()):
        if c == 0:
            continue
        first = c - n  # position of the first query token
        lo = max(0, first - w + 1) if w else 0
        keys += c - lo
        ends = np.arange(first, c) + 1
        pairs += int((ends - (np.maximum(0, ends - w) if w else 0)).sum())
    return keys, pairs


def work(case):
    op = case["op"]
    if op == "linear":
        m, k, n, g = case["rows"], case["n_in"], case["n_out"], case["group"]
        e = _BYTES[case["dtype"]]
        groups = -(-k // g)
        size = n * -(-k // 8) * 4 + n * groups * (3 if case["zeros"] else 2) + (4 * n if case["bias"] else 0)
        return {"bytes": size + m * k * e + m * n * e, "flops": 2 * m * n * k}
    if op == "attend":
        keys, pairs = _visible(case)
        _, q = _lengths(case)
        d, e = case["dim"], _BYTES[case["dtype"]]
        row = d // 2 + 4 * -(-d // case["group"])
        return {"bytes": keys * case["kv_heads"] * 2 * row + 2 * int(q.sum()) * case["heads"] * d * e,
                "flops": 4 * pairs * case["heads"] * d}
    if op == "append":
        d, e = case["dim"], _BYTES[case["dtype"]]
        rows = 2 * case["tokens"] * case["kv_heads"]
        # read, write codes and scales, write the values they stand for
        return {"bytes": rows * (2 * d * e + d // 2 + 4 * -(-d // case["group"])) + 4 * case["tokens"],
                "flops": 8 * rows * d}
    ctx, new = _lengths(case)
    bs = case["block"]
    added = int((-(-(ctx + new) // bs) - -(-ctx // bs)).sum())
    total = int(new.sum())
    return {"bytes": 4 * (3 * case["requests"] + 2 * added + 2 * total + min(total, case["requests"])),
            "flops": 4 * total}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _linear_inputs(case, seed):
    """Codes of a normal weight matrix, steps that vary by a factor of three,
    zero points near the middle, activations with a few large channels."""
    g = _gen(seed)
    m, k, n = case["rows"], case["n_in"], case["n_out"]
    groups = -(-k // case["group"])
    codes = (torch.randn((n, k), generator=g, device="cuda").mul_(3.0).add_(7.5).round_().clamp_(0, 15)).to(torch.uint8)
    scales = (torch.rand((n, groups), generator=g, device="cuda") + 0.5).mul_(0.02).to(torch.float16)
    zeros = torch.randint(5, 11, (n, groups), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    bias = torch.randn((n,), generator=g, device="cuda") if case["bias"] else None
    x = torch.randn((m, k), generator=g, device="cuda")
    x *= 1 + 7 * (torch.rand((k,), generator=g, device="cuda") < 0.01)
    return codes, scales, zeros, bias, x.to(_DTYPES[case["dtype"]])


def _words(codes):
    """[n, k] codes as int32 words [n, ceil(k/8)], input i at bits 4 * (i % 8)."""
    n, k = codes.shape
    pad = torch.nn.functional.pad(codes, (0, -k % 8)).view(n, -1, 8)
    lo = (pad[:, :, 0::2] | (pad[:, :, 1::2] << 4)).contiguous()
    return lo.view(torch.int32).view(n, -1)


def _rows(g, tokens, kv_heads, dim, dtype, outliers):
    """New keys or values as slices of a fused projection (a strided view);
    keys have a few channels that are much larger than the rest."""
    x = torch.randn((tokens, 2 * kv_heads, dim), generator=g, device="cuda")
    if outliers:
        x *= 1 + 5 * (torch.rand((2 * kv_heads, dim), generator=g, device="cuda") < 0.03)
    return x.to(dtype)[:, :kv_heads]


def _append_inputs(case, seed):
    g = _gen(seed)
    t = case["tokens"]
    k = _rows(g, t, case["kv_heads"], case["dim"], _DTYPES[case["dtype"]], True)
    v = _rows(g, t, case["kv_heads"], case["dim"], _DTYPES[case["dtype"]], False)
    blocks = -(-t // case["block"]) + 3
    order = torch.randperm(blocks, generator=g, device="cuda")
    pos = torch.arange(t, device="cuda")
    slots = order[pos // case["block"]] * case["block"] + pos % case["block"]
    if t > 20:
        slots[torch.randint(0, t, (t // 16,), generator=g, device="cuda")] = -1  # padding of a captured batch
    return k, v, slots.to(torch.int32), blocks


def _attend_inputs(case, seed):
    """Keys and values of every cached token, a shuffled block table, queries
    that give logits of standard deviation about 1.5."""
    g = _gen(seed)
    ctx, q = _lengths(case)
    bs = case["block"]
    per = -(-ctx // bs)
    width = int(per.max()) + 1
    blocks = int(per.sum()) + 2
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    count = torch.from_numpy(per).cuda()
    first = torch.cumsum(count, 0) - count
    held = col[None] < count[:, None]
    table = torch.where(held, order[(first[:, None] + col[None]).clamp_(max=blocks - 1)], -1).to(torch.int32)
    shape = (blocks * bs, case["kv_heads"], case["dim"])
    # the cache was filled from 16-bit keys and values
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    queries = torch.randn((int(q.sum()), case["heads"], case["dim"]), generator=g, device="cuda").mul_(1.5)
    starts = torch.from_numpy(np.concatenate([[0], np.cumsum(q)])).to(torch.int32).cuda()
    lens = torch.from_numpy(ctx).to(torch.int32).cuda()
    return k, v, table, lens, starts, queries.to(_DTYPES[case["dtype"]]), int(q.max()), blocks


def _tables_inputs(case, seed):
    g = _gen(seed)
    ctx, new = _lengths(case)
    bs = case["block"]
    have = -(-ctx // bs)
    need = -(-(ctx + new) // bs)
    width = int(need.max()) + 1
    blocks = int(need.sum()) + 5
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    count = torch.from_numpy(have).cuda()
    first = torch.cumsum(count, 0) - count
    col = torch.arange(width, device="cuda")
    table = torch.where(col[None] < count[:, None], order[(first[:, None] + col[None]).clamp_(max=blocks - 1)], -1)
    free = order[int(have.sum()):].contiguous()
    as_int = lambda a: torch.from_numpy(a).to(torch.int32).cuda()  # noqa: E731
    head = torch.zeros(1, dtype=torch.int32, device="cuda")
    return table.to(torch.int32), as_int(ctx), as_int(new), free, head, int(new.sum())


# -------------------------------------------------------------- plain forms

def _unpack(words, k):
    shifts = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    return ((words[:, :, None] >> shifts) & 15).view(words.shape[0], -1)[:, :k]


def _plain_linear(s):
    k, g = s["n_in"], s["group"]
    c = _unpack(s["words"], k).float()
    z = s["zeros"].float().repeat_interleave(g, 1)[:, :k] if s["zeros"] is not None else 8.0
    w = (c - z) * s["scales"].float().repeat_interleave(g, 1)[:, :k]
    y = s["x"].float() @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype)


def _quantise(x, group):
    """Codes (uint8), steps and midpoints (fp16) of [..., dim]; a last group
    may be short."""
    d = x.shape[-1]
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=65504.0, neginf=-65504.0).clamp(-65504.0, 65504.0)
    short = -d % group
    lo = torch.nn.functional.pad(x, (0, short), value=math.inf).unflatten(-1, (-1, group)).amin(-1)
    hi = torch.nn.functional.pad(x, (0, short), value=-math.inf).unflatten(-1, (-1, group)).amax(-1)
    step = ((hi - lo) * (1.0 / 15.0)).half()
    s = step.float()
    mid = (lo + 8.0 * s).half()
    r = torch.where(s > 0, torch.reciprocal(s), 0.0)
    wide = lambda t: t.repeat_interleave(group, -1)[..., :d]  # noqa: E731
    c = (torch.round((x - wide(mid.float())) * wide(r)) + 8.0).clamp_(0, 15)
    return c.to(torch.uint8), step, mid


def _values(c, step, mid, group):
    d = c.shape[-1]
    wide = lambda t: t.float().repeat_interleave(group, -1)[..., :d]  # noqa: E731
    return (c.float() - 8.0) * wide(step) + wide(mid)


def _nibbles(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _from_nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _plain_side(x, slots, codes, steps, mids, group):
    c, step, mid = _quantise(x, group)
    keep = torch.where(slots >= 0, slots, codes.shape[0] - 1).long()  # the last row takes what has no slot
    codes[keep] = _nibbles(c)
    steps[keep] = step
    mids[keep] = mid
    return _values(c, step, mid, group).to(x.dtype)


def _plain_append(s):
    return {"k": _plain_side(s["k"], s["slots"], *s["k_cache"], s["group"]),
            "v": _plain_side(s["v"], s["slots"], *s["v_cache"], s["group"])}


def _plain_attend(s):
    table, lens, starts, q = s["table"], s["lens"].long(), s["starts"].long(), s["q"]
    bs, group, hkv, max_q = s["block"], s["group"], s["kv_heads"], s["max_q"]
    n, dim = table.shape[0], q.shape[-1]
    ratio = q.shape[1] // hkv
    pos = torch.arange(int(s["longest"]), device=q.device)
    slot = table[:, pos // bs].long().clamp_(min=0) * bs + pos % bs                       # [n, L]
    k = _values(_from_nibbles(s["k_cache"][0][slot]), s["k_cache"][1][slot], s["k_cache"][2][slot], group)
    count = starts[1:] - starts[:-1]
    j = torch.arange(max_q, device=q.device)
    row = (starts[:-1, None] + j).clamp_(max=q.shape[0] - 1)                              # [n, max_q]
    qp = q[row].float().view(n, max_q, hkv, ratio, dim).permute(0, 2, 3, 1, 4).reshape(n, hkv, ratio * max_q, dim)
    sc = (qp @ k.permute(0, 2, 3, 1)).view(n, hkv, ratio, max_q, -1) * s["scale"]
    del k
    at = (lens - count)[:, None] + j                                                      # query positions
    seen = (pos <= at[..., None]) & (pos < lens[:, None, None])
    if s["window"]:
        seen &= pos > at[..., None] - s["window"]
    sc = sc.masked_fill_(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top > -math.inf, top, 0.0))
    del sc
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total > 0, total, 1.0)
    v = _values(_from_nibbles(s["v_cache"][0][slot]), s["v_cache"][1][slot], s["v_cache"][2][slot], group)
    o = p.view(n, hkv, ratio * max_q, -1) @ v.permute(0, 2, 1, 3)
    o = o.view(n, hkv, ratio, max_q, dim).permute(0, 3, 1, 2, 4).reshape(n * max_q, hkv * ratio, dim)
    return o[(j < count[:, None]).flatten()].to(q.dtype)


def _plain_tables(s):
    table, ctx, new, bs = s["table"], s["ctx"].long(), s["new"].long(), s["block"]
    total = s["total"]
    have, after = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    added = after - have
    first = s["head"].long() + torch.cumsum(added, 0) - added
    col = torch.arange(table.shape[1], device=table.device)
    fresh = (col >= have[:, None]) & (col < after[:, None])
    source = (first[:, None] + col - have[:, None]).clamp_(0, s["free"].shape[0] - 1)
    table.copy_(torch.where(fresh, s["free"][source], table))
    starts = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    owner = torch.repeat_interleave(torch.arange(ctx.shape[0], device=ctx.device), new, output_size=total)
    pos = ctx[owner] + torch.arange(total, device=ctx.device) - starts[owner]
    slots = table[owner, pos // bs] * bs + (pos % bs).to(torch.int32)
    return {"table": table, "slots": slots, "positions": pos.to(torch.int32), "starts": starts.to(torch.int32),
            "lens": (ctx + new).to(torch.int32), "head": (s["head"] + added.sum()).to(torch.int32)}


# ------------------------------------------------------------- prepare and run

def _plain_cache(rows, kv_heads, dim, group):
    groups = -(-dim // group)
    return (torch.zeros((rows, kv_heads, dim // 2), dtype=torch.uint8, device="cuda"),
            torch.zeros((rows, kv_heads, groups), dtype=torch.float16, device="cuda"),
            torch.zeros((rows, kv_heads, groups), dtype=torch.float16, device="cuda"))


def prepare(case, seed):
    op = case["op"]
    s = {"op": op}
    if op == "linear":
        codes, scales, zeros, bias, x = _linear_inputs(case, seed)
        words = _words(codes)
        s.update(x=x, group=case["group"], n_in=case["n_in"])
        if own:
            import popcount_convolution_amd as pca
            host = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
            s["layer"] = pca.Q4Linear(in_features=case["n_in"], out_features=case["n_out"], group=case["group"],
                                      weight_words=host(words).view(np.uint32), scales=host(scales),
                                      zeros=host(zeros), bias=host(bias))
        else:
            s.update(words=words, scales=scales, zeros=zeros, bias=bias)
        return s
    if op == "append":
        k, v, slots, blocks = _append_inputs(case, seed)
        s.update(k=k, v=v, slots=slots, group=case["group"])
        if own:
            import popcount_convolution_amd as pca
            s["cache"] = pca.KV4Cache(blocks, case["block"], case["kv_heads"], case["dim"], group=case["group"])
        else:
            rows = blocks * case["block"] + 1
            s["k_cache"] = _plain_cache(rows, case["kv_heads"], case["dim"], case["group"])
            s["v_cache"] = _plain_cache(rows, case["kv_heads"], case["dim"], case["group"])
        return s
    if op == "attend":
        k, v, table, lens, starts, q, max_q, blocks = _attend_inputs(case, seed)
        s.update(table=table, lens=lens, starts=starts, q=q, max_q=max_q, scale=1.0 / math.sqrt(case["dim"]),
                 window=case["window"], block=case["block"], group=case["group"], kv_heads=case["kv_heads"],
                 longest=int(_lengths(case)[0].max()))
        if own:
            import popcount_convolution_amd as pca
            s["cache"] = pca.KV4Cache(blocks, case["block"], case["kv_heads"], case["dim"], group=case["group"])
            s["cache"].append(k, v, torch.arange(k.shape[0], dtype=torch.int32, device="cuda"))
        else:
            for name, x in (("k_cache", k), ("v_cache", v)):
                c, step, mid = _quantise(x, case["group"])
                s[name] = (_nibbles(c), step, mid)
        return s
    table, ctx, new, free, head, total = _tables_inputs(case, seed)
    s.update(table=table, ctx=ctx, new=new, free=free, head=head, total=total, block=case["block"])
    return s


def run(state):
    s = state
    op = s["op"]
    if not own:
        return {"linear": _plain_linear, "append": _plain_append, "attend": _plain_attend,
                "tables": _plain_tables}[op](s)
    import popcount_convolution_amd as pca
    if op == "linear":
        return s["layer"].forward(s["x"])
    if op == "append":
        k, v = s["cache"].append(s["k"], s["v"], s["slots"], values=True)
        return {"k": k, "v": v}
    if op == "attend":
        return s["cache"].attention(s["q"], s["table"], s["lens"], scale=s["scale"], window=s["window"],
                                    q_start=s["starts"] if s["max_q"] > 1 else None, max_q=s["max_q"])
    t = pca.build_block_tables(s["table"], s["ctx"], s["new"], s["free"], s["head"], block_size=s["block"],
                               tokens=s["total"])
    return {"table": s["table"], "slots": t.slots, "positions": t.positions, "starts": t.q_start,
            "lens": t.context_lens, "head": t.free_head}


# ----------------------------------------------- the definition, in 64 bits

def _exact_rows(t, group):
    """Cache values of [..., dim] by the format's own steps: every operation in
    64 bits, then rounded to fp32 (or fp16) where the format says so."""
    f32 = lambda a: a.float().double()  # noqa: E731
    f16 = lambda a: a.float().half().double()  # noqa: E731
    fifteenth = float(np.float32(1.0 / 15.0))
    x = t.double()
    out = torch.empty_like(x)
    for at in range(0, x.shape[-1], group):
        part = x[..., at:at + group]
        lo, hi = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
        s = f16(f32(f32(hi - lo) * fifteenth))
        b = f16(f32(lo + 8.0 * s))
        r = torch.where(s > 0, f32(1.0 / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(s))
        c = (f32(f32(part - b) * r).round() + 8.0).clamp(0.0, 15.0)
        out[..., at:at + group] = s * (c - 8.0) + b
    return out


def _exact_linear(case, seed):
    codes, scales, zeros, bias, x = _linear_inputs(case, seed)
    k, n, g = case["n_in"], case["n_out"], case["group"]
    y = torch.zeros((case["rows"], n), dtype=torch.float64, device="cuda")
    for at in range(0, k, g):  # one group of inputs at a time: s * (sum x c - z sum x)
        end = min(k, at + g)
        xs = x[:, at:end].double()
        dot = torch.matmul(xs, codes[:, at:end].double().t().contiguous())
        z = zeros[:, at // g].double() if zeros is not None else 8.0
        y += scales[:, at // g].double() * (dot - z * xs.sum(1, keepdim=True))
    return y + bias.double() if bias is not None else y


def _exact_attend(case, seed):
    k, v, table, lens, starts, q, _, _ = _attend_inputs(case, seed)
    kx, vx = _exact_rows(k, case["group"]), _exact_rows(v, case["group"])
    ctx, count = _lengths(case)
    bs, ratio = case["block"], case["heads"] // case["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    at = 0
    for i in range(case["requests"]):
        length, n = int(ctx[i]), int(count[i])
        pos = torch.arange(length, device="cuda")
        slot = table[i, pos // bs].long() * bs + pos % bs
        where = length - n + torch.arange(n, device="cuda")
        seen = pos[None] <= where[:, None]
        if case["window"]:
            seen &= where[:, None] - pos[None] < case["window"]
        for h in range(case["heads"]):
            if length == 0:
                continue
            kh, vh = kx[slot, h // ratio].contiguous(), vx[slot, h // ratio].contiguous()
            z = torch.matmul(q[at:at + n, h].double(), kh.t().contiguous()) / math.sqrt(case["dim"])
            w = torch.softmax(torch.where(seen, z, torch.full_like(z, -math.inf)), 1)
            out[at:at + n, h] = torch.matmul(w, vh)
        at += n
    return out


def exact(case, seed):
    if case["op"] == "linear":
        return _exact_linear(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, seed)
    if case["op"] == "append":
        k, v, _, _ = _append_inputs(case, seed)
        return {"k": _exact_rows(k, case["group"]), "v": _exact_rows(v, case["group"])}
    return None  # whole numbers only
