"""The decoding example (examples/q4_decode.py): the operators together, as a
server runs them, against the same model in plain 64-bit arithmetic."""

import os
import sys

import numpy as np
import pytest
import torch

import q4_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def plain_weights(host, group):
    codes, scales, zeros = host
    wide = lambda a: np.repeat(a.astype(np.float64), group, 1)[:, :codes.shape[1]]  # noqa: E731
    return wide(scales) * (codes - wide(zeros))


def plain_norm(x):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)


def signs(bits, k):
    b = np.unpackbits(np.ascontiguousarray(bits).view(np.uint8), axis=-1, bitorder="little")
    return b.reshape(bits.shape[0], -1)[:, :k].astype(np.float64) * 2 - 1


def plain_logits(model, tokens):
    """Logits of every position of one sequence; keys and values go through the
    cache's format."""
    c = model.config
    x = model.embedding.double().cpu().numpy()[tokens]
    n, ratio = len(tokens), c.heads // c.kv_heads
    for layer in model.layers:
        qkv = (plain_norm(x) @ plain_weights(layer.host["qkv"], c.group).T).reshape(n, -1, c.head_dim)
        q, k, v = qkv[:, :c.heads], qkv[:, c.heads:c.heads + c.kv_heads], qkv[:, c.heads + c.kv_heads:]
        k, v = (ref.quantise(a.astype(np.float32), c.group)[3].astype(np.float64) for a in (k, v))
        a = np.zeros((n, c.heads, c.head_dim))
        for h in range(c.heads):
            z = q[:, h] @ k[:, h // ratio].T * c.head_dim ** -0.5
            z[np.triu_indices(n, 1)] = -np.inf
            p = np.exp(z - z.max(-1, keepdims=True))
            a[:, h] = p / p.sum(-1, keepdims=True) @ v[:, h // ratio]
        x = x + a.reshape(n, -1) @ plain_weights(layer.host["out"], c.group).T
        up = np.maximum(plain_norm(x) @ signs(layer.up_bits, c.hidden).T * layer.up_scale, 0)
        x = x + up @ signs(layer.down_bits, c.ffn).T * layer.down_scale
    return plain_norm(x) @ plain_weights(model.head_host, c.group).T


def test_weight_quantiser():
    """Weights come back within half a step (and the fp16 rounding of the
    scale), zero exactly."""
    import q4_decode
    rng = np.random.default_rng(0)
    w = rng.normal(0, 1, (7, 100)).astype(np.float32)
    w[:, 3] = 0
    host = q4_decode.quantise_weights(w, 32)
    back = plain_weights(host, 32)
    step = np.repeat(host[1].astype(np.float64), 32, 1)[:, :100]
    assert (np.abs(back - w) <= step * (1 + 15 * 2.0 ** -11)).all()
    assert not back[:, 3].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,bound", [(torch.float32, 0.02), (torch.bfloat16, 0.1)])
def test_decode_matches_plain_model(dtype, bound):
    """Prompts in one chunk, then single tokens: the logits of every step equal
    those of the plain model run over the whole sequence.  A value at a rounding
    boundary of the cache's format may take the neighbouring code, a step of
    1/15 of its group's range; the bounds are well above what a few such steps
    and the activations' rounding give, and far below what a wrong token,
    position or head would (about 1)."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import q4_decode
    model = q4_decode.Model(q4_decode.Config(dtype=dtype), seed=3)
    rng = np.random.default_rng(4)
    prompts = [rng.integers(0, model.config.vocab, n).tolist() for n in (1, 37, 16, 50)]
    session = q4_decode.Session(model, len(prompts), max_blocks=8)
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    got = [[] for _ in prompts]
    first = session.step(torch.tensor(sum(prompts, []), device="cuda"), lens, 50)
    at = 0
    for i, p in enumerate(prompts):
        got[i].append(first[at:at + len(p)])
        at += len(p)
    following = rng.integers(0, model.config.vocab, (20, len(prompts)))
    for row in following:
        y = session.step(torch.from_numpy(row).cuda(), torch.ones_like(lens), 1)
        for i in range(len(prompts)):
            got[i].append(y[i:i + 1])
    assert session.lens.tolist() == [len(p) + 20 for p in prompts]
    for i, p in enumerate(prompts):
        want = plain_logits(model, p + following[:, i].tolist())
        have = torch.cat(got[i]).double().cpu().numpy()
        assert have.shape == want.shape
        rel = np.linalg.norm(have - want, axis=1) / np.linalg.norm(want, axis=1)
        print(f"request {i}: relative error {rel.max():.2e}", flush=True)
        assert rel.max() < bound


@pytest.mark.gpu
def test_generate():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import q4_decode
    model = q4_decode.Model()
    session = q4_decode.Session(model, 2, max_blocks=8)
    out = session.generate([[1, 2, 3], list(range(20))], 5)
    assert out.shape == (2, 5) and session.lens.tolist() == [7, 24]
