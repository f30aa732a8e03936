"""A decoder whose weights and whose key/value cache are both held in blockwise codes: a batch of
ragged prompts enters the cache, then every sequence is continued token by token, the step
captured in a HIP graph.

    python examples/paged_decode.py [--seqs 4] [--prompt 600] [--steps 64] [--layers 4] [--bits 4]

Weights and tokens are random: what is shown is how the calls fit together.  Each layer

    quantized projection -> q, k, v       bq_gemm_blockwise / bq_linear_blockwise
    k, v of the new tokens -> cache       bq_kv_write
    attention of q over the cache         bq_kv_attention
    output projection, gated MLP          bq_gemm_blockwise / bq_linear_blockwise

and at the end one sequence's keys and values are taken out of the cache again (bq_kv_read), and
the last step's attention is compared with the same sums over them in binary64.
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import numpy as np
import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dequantization_block_absmax_amd as bq  # noqa: E402

BLOCK = 64


def table(bits: int) -> np.ndarray:
    """Codes for normally distributed values (4 bits), evenly spaced ones (8 bits)."""
    if bits == 8:
        return np.linspace(-1.0, 1.0, 256).astype(np.float32)
    p = (np.arange(16) + 0.5) / 16
    q = torch.special.ndtri(torch.from_numpy(p)).numpy()
    return (q / np.abs(q).max()).astype(np.float32)


class Linear:
    """y = x W^T with W in 4-bit codes; binary32 out."""

    def __init__(self, n_in, n_out, gen, dev):
        self.n_in, self.n_out = n_in, n_out
        w = torch.randn(n_out, n_in, generator=gen, device=dev, dtype=torch.bfloat16) / math.sqrt(n_in)
        self.table = bq.code_table(table(4))
        self.absmax = torch.empty(bq.num_blocks(w.numel(), BLOCK), device=dev)
        self.packed = torch.empty(bq.packed_bytes(w.numel(), 16), dtype=torch.uint8, device=dev)
        bq.check(bq.bq_quantize_blockwise(w, bq.BQ_BF16, w.numel(), BLOCK, self.table, self.absmax, self.packed),
                 "quantize")

    def __call__(self, x):
        y = torch.empty(x.shape[0], self.n_out, device=x.device)
        call = bq.bq_linear_blockwise if x.shape[0] <= 4 else bq.bq_gemm_blockwise
        bq.check(call(x, bq.BQ_BF16, x.shape[0], self.n_in, self.n_out, BLOCK, self.table, self.absmax, self.packed,
                      y), "linear")
        return y


class Cache:
    """One layer's pool."""

    def __init__(self, bits, pages, page_size, kv_heads, head_dim, dev):
        n = pages * page_size * kv_heads * head_dim
        self.packed = [torch.zeros(n * bits // 8, dtype=torch.uint8, device=dev) for _ in range(2)]
        self.absmax = [torch.zeros(n // BLOCK, device=dev) for _ in range(2)]
        self.c = bq.kv_cache(self.packed[0], self.absmax[0], self.packed[1], self.absmax[1], table(bits), pages,
                             page_size, kv_heads, head_dim, BLOCK)

    def bytes(self):
        return sum(t.numel() * t.element_size() for t in self.packed + self.absmax)


class Batch:
    """The sequences of a call: new tokens, their positions, and the places they take in the cache."""

    def __init__(self, model, q_len, kv_len):
        dev = model.dev
        seq = torch.repeat_interleave(torch.arange(len(q_len)), torch.tensor(q_len)).to(dev)
        start = np.concatenate(([0], np.cumsum(q_len)))
        self.q_start = torch.tensor(start, dtype=torch.int32, device=dev)
        self.kv_len = torch.tensor(kv_len, dtype=torch.int32, device=dev)
        first = torch.tensor([kv - n - s for kv, n, s in zip(kv_len, q_len, start)], device=dev)
        self.seq, self.positions = seq, torch.arange(start[-1], device=dev) + first[seq]
        self.last = self.q_start[1:].long() - 1
        # the longest context there will be: the plan of the captured step holds for every replay
        self.b = bq.kv_batch(self.q_start, self.kv_len, model.pages, int(start[-1]), max(q_len), model.capacity)
        need = bq.bq_kv_attention_workspace_bytes(model.caches[0].c, self.b, bq.BQ_BF16, model.heads)
        self.workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        self.slots = model.slots(seq, self.positions)

    def advance(self, model):
        """The next token of every sequence (of a batch of single tokens), in place: a captured
        step reads the same tensors."""
        self.kv_len += 1
        self.positions += 1
        self.slots.copy_(model.slots(self.seq, self.positions))


class Model:
    def __init__(self, args, dev):
        gen = torch.Generator(device=dev).manual_seed(args.seed)
        self.dev, self.page_size, self.bits = dev, args.page_size, args.bits
        self.dim, self.heads, self.kv_heads, self.head_dim, self.hidden = 512, 8, 2, 128, 1024
        self.rows = (self.heads + 2 * self.kv_heads) * self.head_dim
        self.capacity = args.prompt + args.steps + 8
        per_seq = -(-self.capacity // self.page_size)
        # pages of a sequence lie anywhere in the pool
        order = torch.randperm(args.seqs * per_seq, generator=torch.Generator().manual_seed(args.seed))
        self.pages = order.to(torch.int32).view(args.seqs, per_seq).to(dev)
        self.caches = [Cache(args.bits, args.seqs * per_seq, self.page_size, self.kv_heads, self.head_dim, dev)
                       for _ in range(args.layers)]
        self.embed = torch.randn(args.vocab, self.dim, generator=gen, device=dev, dtype=torch.bfloat16)
        self.layers = [dict(qkv=Linear(self.dim, self.rows, gen, dev),
                            out=Linear(self.heads * self.head_dim, self.dim, gen, dev),
                            up=Linear(self.dim, 2 * self.hidden, gen, dev),
                            down=Linear(self.hidden, self.dim, gen, dev)) for _ in range(args.layers)]
        self.head = Linear(self.dim, args.vocab, gen, dev)
        self.inv = 10000.0 ** (-torch.arange(self.head_dim // 2, device=dev) / (self.head_dim // 2))

    def slots(self, seq, positions):
        return self.pages[seq, positions // self.page_size].long() * self.page_size + positions % self.page_size

    def norm(self, x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def rotate(self, qkv, positions):
        """Rotary positions for q and k, in place."""
        n = self.heads + self.kv_heads
        x = qkv[:, :n * self.head_dim].view(-1, n, 2, self.head_dim // 2)
        angle = positions[:, None, None] * self.inv
        c, s = angle.cos(), angle.sin()
        x0, x1 = x[:, :, 0].clone(), x[:, :, 1].clone()
        x[:, :, 0] = x0 * c - x1 * s
        x[:, :, 1] = x1 * c + x0 * s

    def forward(self, tokens, batch):
        """Logits of every sequence's last token; self.last_q and self.last_out are the last layer's."""
        x = self.embed[tokens].float()
        k_at, v_at = self.heads * self.head_dim, (self.heads + self.kv_heads) * self.head_dim
        for layer, cache in zip(self.layers, self.caches):
            qkv = layer["qkv"](self.norm(x))
            self.rotate(qkv, batch.positions)
            qkv = qkv.to(torch.bfloat16)  # q, k and v are columns of it: strided rows of one tensor
            bq.check(bq.bq_kv_write(cache.c, bq.BQ_BF16, qkv[:, k_at:], qkv[:, v_at:], len(tokens), self.rows,
                                    self.rows, batch.slots), "write")
            o = torch.empty(len(tokens), self.heads * self.head_dim, dtype=torch.bfloat16, device=self.dev)
            bq.check(bq.bq_kv_attention(cache.c, batch.b, bq.BQ_BF16, qkv, self.rows, self.heads,
                                        self.head_dim ** -0.5, 1, 0, o, o.stride(0), None, batch.workspace),
                     "attention")
            self.last_q, self.last_out = qkv, o
            x = x + layer["out"](o)
            gate, up = layer["up"](self.norm(x)).chunk(2, -1)
            x = x + layer["down"]((F.silu(gate) * up).to(torch.bfloat16))
        return self.head(self.norm(x[batch.last]))


def attention_error(model, batch, seq):
    """The last layer's last attention of one sequence's newest token, against binary64 sums over
    the keys and values read back from the cache: the largest difference, relative to the largest
    value."""
    cache, kv = model.caches[-1], int(batch.kv_len[seq])
    slots = model.slots(seq, torch.arange(kv, device=model.dev))
    k, v = (torch.empty(kv, model.kv_heads * model.head_dim, device=model.dev) for _ in range(2))
    bq.check(bq.bq_kv_read(cache.c, bq.BQ_F32, k, v, kv, k.stride(0), v.stride(0), slots), "read")
    row = int(batch.last[seq])
    q = model.last_q[row, :model.heads * model.head_dim].double().cpu().view(model.kv_heads, -1, model.head_dim)
    k, v = (t.double().cpu().view(kv, model.kv_heads, model.head_dim).transpose(0, 1) for t in (k, v))
    p = torch.softmax(q @ k.transpose(1, 2) * model.head_dim ** -0.5, -1)
    got = model.last_out[row].double().cpu().view(model.kv_heads, -1, model.head_dim)
    return float((got - p @ v).abs().max() / v.abs().max())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("seqs", 4), ("prompt", 600), ("steps", 64), ("layers", 4), ("bits", 4), ("page-size", 16),
                        ("vocab", 4096), ("seed", 0)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--eager", action="store_true", help="every step call by call, no graph")
    args = ap.parse_args(argv)
    if args.steps < 2 or args.seqs < 1 or args.prompt < 1:
        ap.error("at least one sequence, one token of prompt and two steps")
    dev = torch.device("cuda:0")
    model = Model(args, dev)

    # ragged prompts, all in one call
    rng = np.random.default_rng(args.seed)
    lens = [args.prompt] + [int(n) for n in rng.integers(1, args.prompt + 1, args.seqs - 1)]
    prompt = torch.from_numpy(rng.integers(0, args.vocab, sum(lens))).to(dev)
    logits = model.forward(prompt, Batch(model, lens, lens))

    # the decoding step, captured once and replayed; its tokens and lengths live on the device
    step = Batch(model, [1] * args.seqs, [n + 1 for n in lens])
    tokens = logits.argmax(-1)
    chosen = []

    def one():
        tokens.copy_(model.forward(tokens, step).argmax(-1))

    one()  # the first step as it is, which also warms every kernel up
    chosen.append(tokens.clone())
    step.advance(model)
    if args.eager:
        replay = one
    else:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            one()
        replay = graph.replay
    torch.cuda.synchronize()
    start = time.perf_counter()
    for i in range(args.steps - 1):
        if i:
            step.advance(model)
        replay()
        chosen.append(tokens.clone())
    torch.cuda.synchronize()
    seconds = time.perf_counter() - start

    errors = [attention_error(model, step, s) for s in range(args.seqs)]
    held = sum(c.bytes() for c in model.caches)
    plain = sum(2 * c.packed[0].numel() * 8 // args.bits * 2 for c in model.caches)
    print(f"{args.seqs} sequences of {min(lens)} to {max(lens)} tokens, {args.layers} layers: "
          f"cache {held / 2**20:.1f} MiB ({plain / held:.2f} times smaller than in bfloat16), "
          f"{seconds / (args.steps - 1) * 1e6:.0f} us a step of the batch, "
          f"attention within {max(errors):.1e} of binary64 over the cached values")
    return torch.stack(chosen, 1), max(errors)


if __name__ == "__main__":
    main()
