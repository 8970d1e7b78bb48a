"""Plain 64-bit references of the microscaled 4-bit operators and of the
experts' order, from the definitions in include/bconv_mx4.h, and bounds of
what fp32 sums and one rounding may differ from them by."""

import numpy as np

MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
PAD, BLOCK = 256, 32
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}  # step of the subnormal numbers


def padded(cols):
    return -(-cols // PAD) * PAD


def quantise(x):
    """(codes [rows, padded / 2], scale bytes [rows, padded / 32], values [rows, cols]) of float64 rows."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    wide = np.zeros((rows, padded(cols)))
    wide[:, :cols] = x
    blocks = wide.reshape(rows, padded(cols) // BLOCK, BLOCK)
    finite = np.isfinite(blocks).all(-1)
    top = np.where(finite, np.abs(np.where(np.isfinite(blocks), blocks, 0)).max(-1), 0)
    _, e = np.frexp(top)                              # top is in [2^(e-1), 2^e)
    e = np.where(top > 0, np.maximum(e - 3, -127), -127)
    q = np.where(finite[..., None], np.ldexp(np.where(finite[..., None], blocks, 0), -e[..., None]), 0)
    index = np.zeros(q.shape, np.int64)
    for i in range(7):
        middle = (MAGNITUDES[i] + MAGNITUDES[i + 1]) / 2
        index += np.abs(q) >= middle if i % 2 else np.abs(q) > middle   # a tie goes to the even code
    code = np.where(finite[..., None], index | (np.signbit(q) << 3), 0).reshape(wide.shape).astype(np.uint8)
    values = np.ldexp(np.copysign(MAGNITUDES[index], q), e[..., None])
    values = np.where(finite[..., None], values, np.nan).reshape(wide.shape)[:, :cols]
    byte = np.where(finite, e + 127, 255).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte, values


def dense(codes, scales, cols):
    """float64 [rows, cols] of packed codes [rows, >= cols / 2] and scale bytes."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)[:, :cols]
    v = np.where(c >= 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    s = np.repeat(scales, BLOCK, 1)[:, :cols].astype(np.int64)
    return np.where(s == 255, np.nan, np.ldexp(v, np.minimum(s, 254) - 127))


def random_weights(rng, rows, cols, low=118, high=122):
    """Codes [rows, ceil(cols / 2)], with whatever in an unused last half, and scale bytes."""
    codes = rng.integers(0, 256, (rows, -(-cols // 2))).astype(np.uint8)
    return codes, rng.integers(low, high, (rows, -(-cols // BLOCK))).astype(np.uint8)


def linear(x, codes, scales, bias):
    """(y, mass): the product of quantised float64 rows x, and the sum of its terms' magnitudes."""
    q, w = quantise(x)[2], dense(codes, scales, x.shape[1])
    y, mass = q @ w.T, np.abs(q) @ np.abs(w).T
    return (y, mass) if bias is None else (y + bias, mass + np.abs(bias))


def linear_bound(y, mass, cols, dtype):
    """Products are exact.  A sum passes at most one addition to its running
    value per 128 values, 31 more where up to 16 waves and 16 parts are joined,
    and one for a bias; an addition of the matrix cores may cut off instead of
    rounding and aligns its terms to the largest, so counts as two steps of 2^-23 of the mass.  Then
    the result is rounded once."""
    additions = -(-cols // 128) + 32
    return 2 * additions * 2.0 ** -23 * mass + HALF_STEP[dtype] * np.abs(y) + LEAST[dtype] / 2


def expert_order(ids, experts):
    """(offsets, order, position) of ids [tokens, choices]."""
    flat = np.asarray(ids).reshape(-1)
    lists = [np.nonzero(flat == e)[0] for e in range(experts)]
    offsets = np.concatenate([[0], np.cumsum([len(i) for i in lists])]).astype(np.int32)
    order = np.full(flat.size, -1, np.int32)
    order[:offsets[-1]] = np.concatenate(lists) if lists else []
    position = np.full(flat.size, -1, np.int32)
    position[order[:offsets[-1]]] = np.arange(offsets[-1])
    return offsets, order, position.reshape(np.shape(ids))
