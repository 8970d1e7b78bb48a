"""Greedy decoding with a small low-bit model: 4-bit projections and cache,
1-bit feed-forward layers.

    python examples/q4_decode.py [--layers 2] [--tokens 16]

A batch of prompts of different lengths goes through the model in one chunk,
then one token a request and step.  Each step is what a server runs:
``build_block_tables`` gives the new tokens their places, ``Q4Linear`` makes
queries, keys and values (one fused projection, whose slices are passed on as
they are), ``KV4Cache.append`` writes the keys and values in 4 bits,
``KV4Cache.attention`` reads them, and the feed-forward layers are the package's
binaryWeights fully connected layers.  Weights are random: the example shows the
calls, not a trained model.
"""

import argparse
import os
import sys
from dataclasses import dataclass

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import popcount_convolution_amd as pca  # noqa: E402


@dataclass
class Config:
    layers: int = 2
    hidden: int = 256
    heads: int = 4
    kv_heads: int = 2
    head_dim: int = 64
    ffn: int = 512
    vocab: int = 500
    group: int = 64
    block_size: int = 16
    num_blocks: int = 256
    dtype: torch.dtype = torch.float32


def quantise_weights(w: np.ndarray, group: int):
    """4-bit codes, fp16 scales and zero points of a float matrix [out, in]:
    per group the range of the values (with 0 in it) in 15 steps."""
    n, k = w.shape
    groups = -(-k // group)
    padded = np.zeros((n, groups * group), np.float32)
    padded[:, :k] = w
    parts = padded.reshape(n, groups, group)
    lo, hi = np.minimum(parts.min(-1), 0), np.maximum(parts.max(-1), 0)
    scales = np.maximum((hi - lo) / 15, 2.0 ** -20).astype(np.float16)
    s = scales.astype(np.float32)
    zeros = np.clip(np.rint(-lo / s), 0, 15).astype(np.uint8)
    codes = np.clip(np.rint(parts / s[..., None]) + zeros[..., None], 0, 15)
    return codes.reshape(n, -1)[:, :k].astype(np.int64), scales, zeros


class Layer:
    """The host weights of one block, and its layers on the GPU."""

    def __init__(self, rng, c: Config):
        rows = (c.heads + 2 * c.kv_heads) * c.head_dim
        self.host = {"qkv": quantise_weights(rng.normal(0, c.hidden ** -0.5, (rows, c.hidden)), c.group),
                     "out": quantise_weights(rng.normal(0, 0.5 * (c.heads * c.head_dim) ** -0.5,
                                                        (c.hidden, c.heads * c.head_dim)), c.group)}
        self.qkv, self.out = (q4_linear(self.host[name], c.group) for name in ("qkv", "out"))
        self.up_bits = rng.integers(0, 2 ** 32, (c.ffn, 1, 1, -(-c.hidden // 32)), dtype=np.uint32)
        self.down_bits = rng.integers(0, 2 ** 32, (c.hidden, 1, 1, -(-c.ffn // 32)), dtype=np.uint32)
        self.up_scale, self.down_scale = c.hidden ** -0.5, 0.5 * c.ffn ** -0.5
        fc = dict(in_h=1, in_w=1, kernel=(1, 1), type="binary_weights")
        self.up = pca.BinaryConvolution(in_c=c.hidden, out_c=c.ffn, weight_bits=self.up_bits,
                                        scale_value=self.up_scale, neuron="relu", **fc)
        self.down = pca.BinaryConvolution(in_c=c.ffn, out_c=c.hidden, weight_bits=self.down_bits,
                                          scale_value=self.down_scale, **fc)


def q4_linear(host, group: int) -> pca.Q4Linear:
    codes, scales, zeros = host
    return pca.Q4Linear(in_features=codes.shape[1], out_features=codes.shape[0], weight_words=pca.pack_codes(codes),
                        scales=scales, zeros=zeros, group=group)


def norm(x):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)


class Model:
    def __init__(self, config: Config = Config(), seed: int = 0):
        c = self.config = config
        rng = np.random.default_rng(seed)
        self.embedding = torch.from_numpy(rng.normal(0, 1, (c.vocab, c.hidden)).astype(np.float32)).cuda()
        self.layers = [Layer(rng, c) for _ in range(c.layers)]
        self.head_host = quantise_weights(rng.normal(0, c.hidden ** -0.5, (c.vocab, c.hidden)), c.group)
        self.head = q4_linear(self.head_host, c.group)


class Session:
    """A batch of requests: one cache a layer, one block table for all."""

    def __init__(self, model: Model, requests: int, max_blocks: int):
        c, self.model = model.config, model
        self.caches = [pca.KV4Cache(c.num_blocks, c.block_size, c.kv_heads, c.head_dim, group=c.group)
                       for _ in model.layers]
        as_int = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((requests, max_blocks), -1, **as_int)
        self.lens = torch.zeros(requests, **as_int)
        self.free = torch.arange(c.num_blocks, **as_int)
        self.head = torch.zeros(1, **as_int)

    def step(self, tokens: torch.Tensor, new_lens: torch.Tensor, max_new: int) -> torch.Tensor:
        """Feeds ``new_lens`` tokens a request (``tokens`` holds them one request
        after the other) and returns the logits of every one."""
        m, c = self.model, self.model.config
        t = pca.build_block_tables(self.table, self.lens, new_lens, self.free, self.head, block_size=c.block_size,
                                   tokens=tokens.numel())
        self.lens, self.head = t.context_lens, t.free_head
        x = m.embedding[tokens]
        for layer, cache in zip(m.layers, self.caches):
            qkv = layer.qkv.forward(norm(x).to(c.dtype)).view(-1, c.heads + 2 * c.kv_heads, c.head_dim)
            q, k, v = qkv.split((c.heads, c.kv_heads, c.kv_heads), 1)
            cache.append(k, v, t.slots)
            a = cache.attention(q, self.table, t.context_lens, q_start=t.q_start, max_q=max_new)
            x = x + layer.out.forward(a.view(-1, c.heads * c.head_dim)).float()
            hidden = layer.up.forward(norm(x).view(-1, 1, 1, c.hidden))
            x = x + layer.down.forward(hidden).view(-1, c.hidden)
        return m.head.forward(norm(x).to(c.dtype)).float()

    def generate(self, prompts, count: int):
        """Greedy continuations of the prompts (lists of token ids)."""
        lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        flat = torch.tensor([t for p in prompts for t in p], device="cuda")
        logits = self.step(flat, lens, max(len(p) for p in prompts))
        last = torch.cumsum(lens, 0) - 1
        token = logits[last].argmax(-1)
        out, ones = [token], torch.ones_like(lens)
        for _ in range(count - 1):
            token = self.step(token, ones, 1).argmax(-1)
            out.append(token)
        return torch.stack(out, 1)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--tokens", type=int, default=16)
    p.add_argument("--bf16", action="store_true", help="bf16 activations (float32 by default)")
    a = p.parse_args()
    model = Model(Config(layers=a.layers, dtype=torch.bfloat16 if a.bf16 else torch.float32))
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, model.config.vocab, n).tolist() for n in (5, 40, 17)]
    session = Session(model, len(prompts), max_blocks=16)
    for prompt, row in zip(prompts, session.generate(prompts, a.tokens).tolist()):
        print(f"{len(prompt)} tokens -> {row}")
    print("cached tokens:", session.lens.tolist(), "blocks used:", session.head.item())


if __name__ == "__main__":
    main()
