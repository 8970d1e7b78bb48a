"""Plain 64-bit references of the 4-bit operators, written from their formulas
(include/bconv_q4.h) in numpy, and the error bounds the tests hold them to."""

import numpy as np

# unit roundoff of each result type: 24, 11 and 8 significant bits
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}  # half an fp16 subnormal step
EPS = 2.0 ** -24


# ----------------------------------------------------------------- linear

def unpack_words(words, k):
    """uint32 words [n, ceil(k/8)] -> codes [n, k]."""
    w = words[:, :, None] >> (4 * np.arange(8, dtype=np.uint32))
    return (w & 15).reshape(words.shape[0], -1)[:, :k]


def linear(x, words, scales, zeros, bias, group):
    """float64 result and the per-element sum of |x| * |s| * 31 the fp32 bound uses."""
    k = x.shape[1]
    c = unpack_words(words, k).astype(np.float64)
    wide = lambda a: np.repeat(a.astype(np.float64), group, 1)[:, :k]  # noqa: E731
    s = wide(scales)
    z = wide(zeros) if zeros is not None else 8.0
    x = x.astype(np.float64)
    y = x @ (s * (c - z)).T + (bias.astype(np.float64) if bias is not None else 0.0)
    return y, np.abs(x) @ (31.0 * np.abs(s)).T


def linear_bound(y, mass, bias, k, group, dtype):
    """Every fp32 rounding of the kernel is of a partial sum no larger than the
    sum of |x| (code + offset <= 31 + 31) |s|: at most two products a weight
    within its group, then one a group and wave, then the join of the waves and
    the bias.  The parts of an fp32 x (up to three) multiply the products of a group."""
    steps = 2 * group * (3 if dtype == "f32" else 1) + -(-k // 32) + 64
    b = np.abs(bias).max() if bias is not None and bias.size else 0.0
    return ROUND[dtype] * (1 + 2.0 ** -8) * np.abs(y) + 2.0 * EPS * steps * (mass + b) + TINY[dtype]


# ------------------------------------------------------------------ cache

def quantise(x, group):
    """The cache format's fp32 steps on float32 x [..., dim]: codes, s, b
    (float16 [..., groups]) and values float32."""
    x = np.asarray(x, np.float32)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-65504), np.float32(65504)))
    d = x.shape[-1]
    groups = -(-d // group)
    codes = np.zeros(x.shape, np.uint8)
    s16 = np.zeros(x.shape[:-1] + (groups,), np.float16)
    b16 = np.zeros_like(s16)
    val = np.zeros_like(x)
    for g in range(groups):
        part = x[..., g * group:(g + 1) * group]
        lo, hi = part.min(-1), part.max(-1)
        s = ((hi - lo) * np.float32(1.0 / 15.0)).astype(np.float16)
        sf = s.astype(np.float32)
        b = (lo + np.float32(8) * sf).astype(np.float16)
        bf = b.astype(np.float32)
        r = np.divide(np.float32(1), sf, out=np.zeros_like(sf), where=sf > 0)
        c = np.clip(np.rint((part - bf[..., None]) * r[..., None]) + np.float32(8), 0, 15)
        codes[..., g * group:(g + 1) * group] = c
        s16[..., g], b16[..., g] = s, b
        val[..., g * group:(g + 1) * group] = sf[..., None] * (c.astype(np.float32) - 8) + bf[..., None]
    return codes, s16, b16, val


def read_pool(pool, layout, num_blocks, block_size, kv_heads, dim):
    """Codes and (s, b) of every row of a pool (uint8 array), from the layout
    documented with bconv_kv4_layout_t: two dicts (keys, values) of codes
    [slots, heads, dim] and s, b [slots, heads, groups]."""
    P, G = layout.dim_padded, layout.groups
    rec = np.asarray(pool).reshape(num_blocks, kv_heads, layout.record_bytes)
    out = []
    for side in ("k", "v"):
        co = 0 if side == "k" else layout.v_codes_offset
        so = layout.k_scales_offset if side == "k" else layout.v_scales_offset
        raw = rec[:, :, co:co + block_size * layout.row_bytes].reshape(num_blocks, kv_heads, block_size, -1)
        codes = np.zeros((num_blocks, kv_heads, block_size, P), np.uint8)
        if side == "k":
            w = np.ascontiguousarray(raw).view(np.uint32)
            w = (w >> np.uint32(3)) | (w << np.uint32(29))
            for a in range(4):
                for s in range(P // 32):
                    for i in range(8):
                        nib = i // 2 + 4 * (i % 2)
                        codes[..., 32 * s + 8 * a + i] = (w[..., a * (P // 32) + s] >> np.uint32(4 * nib)) & 15
        else:
            nibs = np.stack([raw & 15, raw >> 4], -1).reshape(raw.shape[:-1] + (P,))
            for r in range(16):
                for j in range(P // 16):
                    codes[..., 16 * j + r] = nibs[..., r * (P // 16) + j]
        sb = np.ascontiguousarray(rec[:, :, so:so + block_size * G * 4]).view(np.float16)
        sb = sb.reshape(num_blocks, kv_heads, block_size, G, 2)
        rows = lambda a: a.transpose(0, 2, 1, 3).reshape(num_blocks * block_size, kv_heads, -1)  # noqa: E731
        out.append({"codes": rows(codes)[..., :dim], "s": rows(sb[..., 0]), "b": rows(sb[..., 1])})
    return out


# -------------------------------------------------------------- attention

def attention(q, kx, vx, vstep, table, lens, counts, *, block_size, kv_heads, scale, window=0, num_blocks=None):
    """q [T, heads, dim]; kx, vx float64 [slots, kv_heads, dim]; vstep [slots,
    kv_heads] the largest step of a value row.  Returns out, lse and what the
    bound needs: the largest |logit| terms' sum, largest |value|, and
    sum p * step."""
    q = q.astype(np.float64)
    T, heads, dim = q.shape
    ratio = heads // kv_heads
    out = np.zeros(q.shape)
    lse = np.full((T, heads), -np.inf)
    zmass, vmax, pstep = np.zeros((T, heads)), np.zeros((T, heads)), np.zeros((T, heads))
    at = 0
    for r, n in enumerate(counts):
        for j in range(n):
            pos_q = int(lens[r]) - n + j
            lo = max(0, pos_q - window + 1) if window else 0
            pos = np.arange(lo, pos_q + 1)
            entry = pos // block_size
            pos = pos[entry < table.shape[1]]
            block = table[r, pos // block_size]
            keep = (block >= 0) & (block < (num_blocks if num_blocks is not None else 1 << 30))
            slot = block[keep].astype(np.int64) * block_size + pos[keep] % block_size
            for h in range(heads):
                if not slot.size:
                    continue
                k, v = kx[slot, h // ratio], vx[slot, h // ratio]
                z = scale * (k @ q[at, h])
                top = z.max()
                p = np.exp(z - top)
                l = p.sum()
                out[at, h] = (p / l) @ v
                lse[at, h] = top + np.log(l)
                zmass[at, h] = abs(scale) * (np.abs(k) @ np.abs(q[at, h])).max()
                vmax[at, h] = np.abs(v).max()
                pstep[at, h] = (p / l) @ vstep[slot, h // ratio]
            at += 1
    return out, lse, (zmass, vmax, pstep)


def attention_bound(out, terms, dim, longest, dtype):
    """A logit is a sum of dim products over at most 24 (code + offset) steps
    and the midpoints, each partial sum at most 5 times the final terms' (the
    offset of 24 against codes of up to 8 around the middle, plus the
    midpoints): zerr.  Probabilities carry zerr twice (numerator and
    denominator) and the rounding of exp2; they are rounded for the matrix
    cores to parts of 8, 16 or 24 bits together times a code of at most 8 steps, and the value
    sums run with an offset of 136 steps (24 in fp32) in fp32."""
    zmass, vmax, pstep = (t[..., None] for t in terms)
    parts = 3 if dtype == "f32" else 1
    zerr = EPS * (dim * parts + 16) * 8 * zmass
    up = {"bf16": 2.0 ** -8, "f16": 2.0 ** -16, "f32": 2.0 ** -24}[dtype]
    off = 31 if dtype == "f32" else 143
    chain = 32 * parts + longest // 32 + 32
    return (ROUND[dtype] * (1 + 2.0 ** -7) * np.abs(out) + vmax * (4 * zerr + 2.0 ** -20) +
            pstep * (8 * up + EPS * chain * off) + TINY[dtype])


# ------------------------------------------------------------ block tables

def block_tables(table, ctx, new, free, head, block_size, tokens):
    table = table.copy()
    width = table.shape[1]
    slots, positions, starts = [], [], [0]
    taken = head
    for r in range(len(ctx)):
        c, n = max(0, int(ctx[r])), max(0, int(new[r]))
        have, need = -(-c // block_size), min(-(-(c + n) // block_size), width)
        for e in range(have, need):
            table[r, e] = free[taken] if 0 <= taken < len(free) else -1
            taken += 1
        for i in range(n):
            p = c + i
            e = p // block_size
            b = int(table[r, e]) if e < width else -1
            slots.append(b * block_size + p % block_size if b >= 0 else -1)
            positions.append(p)
        starts.append(starts[-1] + n)
    pad = tokens - len(slots)
    slots, positions = (slots + [-1] * pad)[:tokens], (positions + [0] * pad)[:tokens]
    lens = [max(0, int(c)) + max(0, int(n)) for c, n in zip(ctx, new)]
    as_int = lambda a: np.array(a, np.int32)  # noqa: E731
    return dict(table=table, slots=as_int(slots), positions=as_int(positions), q_start=as_int(starts),
                context_lens=as_int(lens), free_head=as_int([taken]))
