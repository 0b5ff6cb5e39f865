"""The attention block of a decoder layer, served in IF4 throughout.

Weights and activations are IF4 operands of if4.gemm (W4A4), keys and values go
into a paged IF4 cache as they are projected, and attention reads them from
there: prompts in chunks, then one token of every sequence at a time, whatever
their lengths.  Rotary embeddings, norms and the rest of a layer are left to
the model around it.

Run: `python -m adaptive_block_scaled_amd.decoder_attention [--hidden 4096
--heads 32 --kv-heads 8 --batch 16 --prompt 2000 --steps 32 --window 0]`
serves synthetic prompts through one block with random weights and prints the
time of the prompt and of a decode step, and how far the block's output is from
the same block with its cache left in bf16.
"""
import argparse
import json

import numpy as np
import torch

from . import if4, kv_cache
from . import workloads as wl

K_LIMIT, V_LIMIT = 48.0, 8.0  # largest |k| and |v| that the cache's exponents are set for


class Pages:
    """Which pages of a cache belong to which sequence (host side)."""

    def __init__(self, pages: int, page_size: int, device):
        self.free, self.size, self.device = list(range(pages))[::-1], page_size, device
        self.owned, self.lens = {}, {}

    def extend(self, seq, tokens: int):
        """Room for `tokens` more of a sequence: their slots, as a list."""
        return self.extend_all([seq], [tokens])

    def extend_all(self, seqs, counts):
        """Room for counts[i] more tokens of seqs[i], all different: their slots, one
        sequence after another.  Where the free pages are too few for all of
        them, none gets any."""
        if len(set(seqs)) != len(seqs):
            raise ValueError("a sequence comes twice")
        missing = [-(-(self.lens.get(s, 0) + n) // self.size) - len(self.owned.get(s, ()))
                   for s, n in zip(seqs, counts)]
        if sum(missing) > len(self.free):
            raise MemoryError("the cache has too few free pages")
        slots = []
        for seq, tokens, more in zip(seqs, counts, missing):
            pages, n = self.owned.setdefault(seq, []), self.lens.get(seq, 0)
            pages += [self.free.pop() for _ in range(more)]
            self.lens[seq] = n + tokens
            slots += [pages[j // self.size] * self.size + j % self.size for j in range(n, n + tokens)]
        return slots

    def release(self, seq):
        self.free += self.owned.pop(seq, [])
        self.lens.pop(seq, None)

    def table(self, seqs):
        """(page_table, seq_lens) of these sequences on the device."""
        width = max(len(self.owned[s]) for s in seqs)
        rows = [self.owned[s] + [0] * (width - len(self.owned[s])) for s in seqs]
        i32 = dict(dtype=torch.int32, device=self.device)
        return torch.tensor(rows, **i32), torch.tensor([self.lens[s] for s in seqs], **i32)


class AttentionBlock:
    def __init__(self, w_qkv: torch.Tensor, w_o: torch.Tensor, heads: int, kv_heads: int,
                 pages: int, page_size: int, window: int = 0, sinks: int = 0):
        """w_qkv [(heads + 2 kv_heads) D, hidden] and w_o [hidden, heads D],
        bf16 on the GPU; quantized once."""
        self.heads, self.kv_heads = heads, kv_heads
        self.dim = w_qkv.shape[0] // (heads + 2 * kv_heads)
        self.window, self.sinks = window, sinks
        self.w_qkv, self.w_o = self._weights(w_qkv), self._weights(w_o)
        self.cache = kv_cache.empty(pages, page_size, kv_heads, self.dim, w_qkv.device)
        self.pages = Pages(pages, page_size, w_qkv.device)
        self.exps = dict(k_exp=wl.tensor_scale_exp(K_LIMIT), v_exp=wl.tensor_scale_exp(V_LIMIT))

    @staticmethod
    def _weights(w):
        exp = wl.tensor_scale_exp(float(w.abs().max()))
        return (*if4.quantize(w, exp), exp)

    @staticmethod
    def _linear(x, w, exp):
        """x W^T with x quantized at exponent `exp`, fp32."""
        return if4.gemm(*if4.quantize(x, exp), exp, *w)

    def forward(self, x: torch.Tensor, seqs, counts, x_exp: int = -8, out_exp: int = -8):
        """x [sum(counts), hidden] bf16: counts[i] new tokens of sequence seqs[i],
        one sequence after another.  x_exp, out_exp: exponents that the two
        products' activations are quantized with.  Returns [sum(counts), hidden]
        fp32."""
        h, kv, d = self.heads, self.kv_heads, self.dim
        qkv = self._linear(x, self.w_qkv, x_exp).view(-1, h + 2 * kv, d)
        slots = self.pages.extend_all(seqs, counts)
        kv_cache.append(self.cache, qkv[:, h:h + kv], qkv[:, h + kv:],
                        torch.tensor(slots, device=x.device), **self.exps)
        table, lens = self.pages.table(seqs)
        starts = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32,
                              device=x.device)
        out = kv_cache.attention(qkv[:, :h].bfloat16(), self.cache, table, lens, starts,
                                 max_q=max(counts), max_len=max(self.pages.lens[s] for s in seqs),
                                 window=self.window, sinks=self.sinks, **self.exps)
        return self._linear(out.view(-1, h * d), self.w_o, out_exp)

    def reference(self, xs, x_exp: int = -8, out_exp: int = -8):
        """The same block on one whole sequence xs [n, hidden], keys and values
        kept as projected, in torch."""
        h, kv, d = self.heads, self.kv_heads, self.dim
        qkv = self._linear(xs, self.w_qkv, x_exp).view(-1, h + 2 * kv, d)
        q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        k, v = (t.repeat_interleave(h // kv, 1).transpose(0, 1).contiguous() for t in (k, v))
        s = torch.matmul(q.transpose(0, 1).contiguous(), k.transpose(1, 2).contiguous()) * d ** -0.5
        i = torch.arange(len(xs), device=xs.device)
        seen = i <= i[:, None]
        if self.window:
            seen &= (i > i[:, None] - self.window) | (i < self.sinks)
        p = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
        out = torch.matmul(p, v).transpose(0, 1).reshape(-1, h * d)
        return self._linear(out.bfloat16().contiguous(), self.w_o, out_exp)


def random_block(hidden, heads, kv_heads, dim, pages, page_size, window=0, sinks=0, seed=0):
    rows = (heads + 2 * kv_heads) * dim
    w = [torch.from_numpy(wl.normal_weights(*shape, seed + i, std=shape[1] ** -0.5)).bfloat16().cuda()
         for i, shape in enumerate(((rows, hidden), (hidden, heads * dim)))]
    return AttentionBlock(*w, heads, kv_heads, pages, page_size, window, sinks)


def serve(block, prompts, steps, chunk, hidden, seed=1):
    """Prompts of these lengths in chunks, then `steps` decode steps of all of
    them.  Returns (inputs per sequence, outputs per sequence, ms of the prompts, ms
    per decode step)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    xs = [torch.randn(n + steps, hidden, generator=g, device="cuda").bfloat16() for n in prompts]
    outs = [[] for _ in prompts]
    mark = [torch.cuda.Event(enable_timing=True) for _ in range(3)]

    def step(done, counts):
        live = [i for i, n in enumerate(counts) if n]
        x = torch.cat([xs[i][done[i]:done[i] + counts[i]] for i in live])
        y = block.forward(x, live, [counts[i] for i in live])
        for i, part in zip(live, y.split([counts[i] for i in live])):
            outs[i].append(part)
            done[i] += counts[i]

    mark[0].record()
    done = [0] * len(prompts)
    while any(d < n for d, n in zip(done, prompts)):
        step(done, [min(chunk, n - d) for d, n in zip(done, prompts)])
    mark[1].record()
    for _ in range(steps):
        step(done, [1] * len(prompts))
    mark[2].record()
    torch.cuda.synchronize()
    return xs, [torch.cat(o) for o in outs], mark[0].elapsed_time(mark[1]), \
        mark[1].elapsed_time(mark[2]) / max(steps, 1)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("hidden", 4096), ("heads", 32), ("kv-heads", 8), ("dim", 128), ("batch", 16),
                        ("prompt", 2000), ("chunk", 512), ("steps", 32), ("page-size", 64),
                        ("window", 0), ("sinks", 0)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args(argv)
    prompts = [max(1, a.prompt - 97 * i) for i in range(a.batch)]
    pages = sum(-(-(n + a.steps) // a.page_size) for n in prompts)
    block = random_block(a.hidden, a.heads, a.kv_heads, a.dim, pages, a.page_size, a.window, a.sinks)
    serve(block, [min(64, n) for n in prompts], 1, a.chunk, a.hidden)  # first launches
    for seq in range(a.batch):
        block.pages.release(seq)
    xs, outs, prompt_ms, step_ms = serve(block, prompts, a.steps, a.chunk, a.hidden)
    want = block.reference(xs[-1])
    far = float((outs[-1] - want).norm() / want.norm())
    c = block.cache
    used = sum(t.numel() for t in c)
    print(json.dumps({"prompt_tokens": sum(prompts), "prompt_ms": round(prompt_ms, 3),
                      "decode_ms_per_step": round(step_ms, 4), "cache_MB": round(used / 1e6, 1),
                      "bf16_cache_MB": round(4 * c.k_codes.numel() * 2 / 1e6, 1),
                      "rel_error_of_the_if4_cache": round(far, 4)}))


if __name__ == "__main__":
    main()
