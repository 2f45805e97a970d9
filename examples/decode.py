"""Decode steps of whole layers: attention over the 8-bit paged cache, then the sparse FFN.

    python examples/decode.py [--layers 8] [--seqs 8] [--prompt 500] [--tokens 64] [--window 0 --sinks 0] [--code e4m3]

Random weights and inputs (there is nothing to decode): each step's output, normalised, is the next step's input.
The prompts go in by pieces; a step (room for a token, then per layer the projections, append, attend and the
FFN) is captured once and replayed.  Then the second half of the sequences gives way to forks of the first, and the pool
is compacted, as a beam search or a server does between steps.
"""

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import activation_sparse_decode_relu_amd as pi  # noqa: E402
from synth import make_layer  # noqa: E402
from synth.configs import LayerConfig  # noqa: E402

PIECE = 32   # tokens of a sequence in a piece of a prompt
BATCH = 64   # tokens of an FFN call


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Decoder:
    """Layers of attention and sparse FFN in fp16: 8 query heads of 128 dims on 2 cached heads."""

    heads, kv_heads, dim = 8, 2, 128

    def __init__(self, layers, seqs, max_tokens, window=0, sinks=0, code="e4m3", page_tokens=64, mode="predicted", seed=0):
        cfg = LayerConfig(name="decoder", cfg_id=9, workload="decoder d=1024 n=4096 r=128", d_model=1024, d_ffn=4096, rank=128,
                          gated=True, w_dtype="f16", p_dtype="f16", act_dtype="f16", n_layers=layers, tokens=1,
                          density=0.10, zipf_s=1.1)
        self.d, self.window, self.sinks, self.seqs, self.mode = cfg.d_model, window, sinks, seqs, mode
        self.ffn, shared = [], None
        for i in range(layers):
            self.ffn.append(pi.upload_layer(make_layer(cfg, i, seed), max_batch=BATCH, workspace=shared))
            shared = self.ffn[0].workspace                 # the layers' calls follow one another
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        width = (self.heads + 2 * self.kv_heads) * self.dim
        self.qkv = [(torch.randn(self.d, width, device="cuda", generator=g) * self.d ** -0.5).half() for _ in range(layers)]
        self.proj = [(torch.randn(self.heads * self.dim, self.d, device="cuda", generator=g) * self.d ** -0.5).half()
                     for _ in range(layers)]
        per_seq = -(-max_tokens // page_tokens)
        self.cache = pi.KVCache(self.heads, self.kv_heads, self.dim, pages=seqs * (per_seq + 1), page_tokens=page_tokens,
                                max_seqs=seqs, max_seq_pages=per_seq, code=code, layers=layers)

    def run(self, x, seqs, counts, starts, max_new):
        """The next counts[i] tokens of seqs[i], rows [starts[i], starts[i + 1]) of x [rows][d], through every layer."""
        rows, h, kv = x.shape[0], self.heads, self.kv_heads
        self.cache.reserve(seqs, counts)
        for i, ffn in enumerate(self.ffn):
            t = (norm(x) @ self.qkv[i]).view(rows, h + 2 * kv, self.dim)
            self.cache.append(i, t[:, h:h + kv], t[:, h + kv:], seqs, starts)
            out = torch.empty(rows, h, self.dim, dtype=x.dtype, device=x.device)
            self.cache.attend(i, t[:, :h], out, seqs, starts, max_new, window=self.window, sinks=self.sinks)
            x = x + out.view(rows, -1) @ self.proj[i]
            y, z = norm(x), torch.empty_like(x)
            for at in range(0, rows, BATCH):
                ffn.forward(y[at:at + BATCH], z[at:at + BATCH], self.mode)
            x = x + z
        return x

    def prompts(self, x):
        """x [seqs][tokens][d], by pieces of PIECE tokens; returns the last token's output of each sequence."""
        n, tokens, _ = x.shape
        seqs = ints(range(n))
        for at in range(0, tokens, PIECE):
            piece = x[:, at:at + PIECE]
            c = piece.shape[1]
            y = self.run(piece.reshape(n * c, -1), seqs, ints([c] * n), ints(range(0, n * c + 1, c)), c)
        return y.view(n, c, -1)[:, -1]

    def capture(self, x):
        """A graph that takes one token of every sequence from x [seqs][d] and puts the output's norm back."""
        n = self.seqs
        self.step_ids = ints(range(n)), ints([1] * n), ints(range(n + 1))   # the graph reads them: they live as long as it
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x.copy_(norm(self.run(x, *self.step_ids, 1)))
        return graph


def ints(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("layers", 8), ("seqs", 8), ("prompt", 500), ("tokens", 64), ("window", 0), ("sinks", 0)):
        p.add_argument(f"--{name}", type=int, default=value)
    p.add_argument("--code", choices=("e4m3", "int8"), default="e4m3")
    a = p.parse_args()
    if not 2 <= a.seqs <= BATCH:
        p.error(f"--seqs must lie in [2, {BATCH}]")
    model = Decoder(a.layers, a.seqs, a.prompt + 2 * a.tokens + 2, a.window, a.sinks, a.code)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(a.seqs, a.prompt, model.d, device="cuda", generator=g).half()
    first = norm(model.prompts(x))
    model.run(first.clone(), ints(range(a.seqs)), ints([1] * a.seqs), ints(range(a.seqs + 1)), 1)   # warms the libraries up
    state = first.clone()
    graph = model.capture(state)

    def steps(count):
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(count):
            graph.replay()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / max(count, 1)

    s = steps(a.tokens)
    print(f"{a.seqs} sequences, {a.layers} layers: {s * 1e6:.0f} us a step, {a.seqs / s:.0f} tokens/s")
    half = a.seqs // 2
    model.cache.free(ints(range(a.seqs - half, a.seqs)))
    model.cache.fork(ints(range(half)), ints(range(a.seqs - half, a.seqs)))
    state[a.seqs - half:] = state[:half] + 0.01 * torch.randn(half, model.d, device="cuda", generator=g).half()
    model.cache.compact()
    used = int((model.cache.refs > 0).sum())
    s = steps(a.tokens)
    model.cache.check_failed()
    assert bool(torch.isfinite(state).all())
    print(f"after the fork: {used} pages held of {model.cache.desc.pages}; {s * 1e6:.0f} us a step, {a.seqs / s:.0f} tokens/s")


if __name__ == "__main__":
    main()
