"""Root-mean-square error bounds of the fp32 4-bit operators, tight enough that an
operand held in one fp16 part instead of two does not pass.

Roundings are taken as independent, so that errors add in squares; every bound
is twice what follows from the largest error of each, for what is not
independent after all.  Unit: u = 2^-24, fp32's.

Linear layer.  A term x w of a result has an error of at most 2u of itself (x in
two fp16 parts: 2^-23), which gives 2u S with S^2 the sum of the squared terms.
Sums are rounded once per matrix instruction (16 terms at least, of each of the
two parts), group, wave or split and bias: N = k/8 + groups + 24 roundings of
partial sums, at most P, the largest prefix sum over the groups, or one group's
own.  Together 2 (2u S + u sqrt(N) P) + u |y|.

Attention.  A logit's error is that of such a sum over the channels, with S and P
both taken as Z = |scale| sqrt(sum q^2 k^2), the largest of the visible tokens' (+ the
rounding of the finished logit and of its distance from the maximum, 4u (|z| + 1)),
and exp2's 2u: dz.  An error e_t of a probability moves the result by p_t e_t (v_t -
o), in squares dz V with V^2 = sum p^2 (v - o)^2.  A probability times its step is
held to 2u (two parts), times a code of at most 8: 2u W with W^2 = sum (8 p s)^2.
The sums over tokens are rounded N = tiles of 32 tokens x 2 + 32 times (waves,
parts) at no more than A = sum p |v|.
Together 2 (dz V + 2u W + u sqrt(N) A) + u |o|; the log-sum-exp has 2 (dz sqrt(sum
p^2) + u sqrt(N)) + 4u (1 + |lse|).
"""

import numpy as np

import q4_reference as ref

U = 2.0 ** -24


def linear(x, words, scales, zeros, bias, group):
    """Result in 64 bits and the bound of each element's rms error."""
    k = x.shape[1]
    x = x.astype(np.float64)
    c = ref.unpack_words(words, k).astype(np.float64)
    wide = lambda a: np.repeat(a.astype(np.float64), group, 1)[:, :k]  # noqa: E731
    w = wide(scales) * (c - (wide(zeros) if zeros is not None else 8.0))
    y = np.zeros((x.shape[0], w.shape[0]))
    most = np.zeros_like(y)
    for g in range(0, k, group):
        part = x[:, g:g + group] @ w[:, g:g + group].T
        y += part
        most = np.maximum(most, np.maximum(np.abs(y), np.abs(part)))
    if bias is not None:
        y += bias.astype(np.float64)
        most = np.maximum(most, np.abs(y))
    terms = np.sqrt((x * x) @ (w * w).T)
    n = k / 8 + -(-k // group) + 24
    return y, 2 * (2 * U * terms + U * np.sqrt(n) * most) + U * np.abs(y)


def attention(q, k, v, step, lens, counts, scale, group):
    """q [T, heads, dim]; k, v [requests][tokens, kv_heads, dim] and step
    [requests][tokens, kv_heads] (the largest of a row) in 64 bits.  Result, log-sum-exp and
    the bounds of their elements' rms errors; no window."""
    q = q.astype(np.float64)
    total, heads, dim = q.shape
    out, lse = np.zeros(q.shape), np.zeros((total, heads))
    bound, lse_bound = np.zeros(q.shape), np.zeros((total, heads))
    n = 2 * (max(lens) / 32) + 32
    nz = dim / 8 + -(-dim // group) + 4
    at = 0
    for r, count in enumerate(counts):
        for j in range(count):
            end = int(lens[r]) - count + j + 1
            for h in range(heads):
                g = h // (heads // k[r].shape[1])
                kk, vv, ss = k[r][:end, g], v[r][:end, g], step[r][:end, g]
                z = scale * (kk @ q[at, h])
                p = np.exp(z - z.max())
                lse[at, h] = z.max() + np.log(p.sum())
                p /= p.sum()
                o = p @ vv
                size = abs(scale) * np.sqrt((kk * kk) @ (q[at, h] ** 2)).max()
                dz = 2 * U * size + U * np.sqrt(nz) * size + 4 * U * (np.abs(z).max() + 1) + 2 * U
                spread = np.sqrt(((p[:, None] * (vv - o)) ** 2).sum(0))
                code = np.sqrt(((8 * p * ss) ** 2).sum())
                out[at, h] = o
                bound[at, h] = 2 * (dz * spread + 2 * U * code + U * np.sqrt(n) * (p @ np.abs(vv))) + U * np.abs(o)
                lse_bound[at, h] = 2 * (dz * np.sqrt((p * p).sum()) + U * np.sqrt(n)) + 4 * U * (1 + abs(lse[at, h]))
            at += 1
    return out, lse, bound, lse_bound


def rms(a):
    return np.sqrt((np.asarray(a, np.float64) ** 2).mean())


def parts(x, count, axis_top):
    """x as `count` fp16 parts after a power of two takes the largest magnitude,
    axis_top, to 2^14."""
    to = 2.0 ** (14 - np.floor(np.log2(axis_top)))
    y = np.asarray(x, np.float64) * to
    h = y.astype(np.float16).astype(np.float64)
    return (h + ((y - h).astype(np.float16) if count == 2 else 0)) / to
