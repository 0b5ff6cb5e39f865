"""The attention block of a decoder layer, served in IF4 throughout, or with its
projections in FP8.

Weights and activations are IF4 operands of if4.gemm (W4A4), or FP8 ones of fp8.gemm
where four bits cost too much; keys and values go into a paged IF4 cache as they are
projected, and attention reads them from there: prompts in chunks, then one token of
every sequence at a time, whatever their lengths.  With a Rotation, queries and keys are
normed for each head and rotated by their positions in between.  A block that keeps
count of attention weights can cut a sequence's cache to the tokens that matter
(evict), and goes on with those.  The rest of a layer is left to the model around it.

Run: `python -m adaptive_block_scaled_amd.decoder_attention [--hidden 4096
--heads 32 --kv-heads 8 --batch 16 --prompt 2000 --steps 32 --window 0
--precision if4 --rotary 0 --keep 0]` serves synthetic prompts through one block with
random weights and prints the time of the prompt and of a decode step, and how far the
block's output is from the same block with its cache left in bf16 (with --keep, after
the prompts' caches have been cut to so many tokens: from the same without a cut).
"""
import argparse
import json
from typing import NamedTuple

import numpy as np
import torch

from . import fp8, if4, kv_cache, kv_evict, qk
from . import workloads as wl

K_LIMIT, V_LIMIT = 48.0, 8.0  # largest |k| and |v| that the cache's exponents are set for


class Pages:
    """Which pages of a cache belong to which sequence (host side)."""

    def __init__(self, pages: int, page_size: int, device):
        self.free, self.size, self.device = list(range(pages))[::-1], page_size, device
        self.owned, self.lens = {}, {}  # of each sequence: its pages, its tokens in them
        self.seen = {}                  # its tokens so far, evicted ones among them

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
            self.seen[seq] = self.seen.get(seq, 0) + tokens
            slots += [pages[j // self.size] * self.size + j % self.size for j in range(n, n + tokens)]
        return slots

    def positions(self, seqs, counts):
        """Positions that counts[i] more tokens of seqs[i] will have, as a list."""
        return [j for s, n in zip(seqs, counts) for j in range(self.seen.get(s, 0), self.seen.get(s, 0) + n)]

    def fresh(self, counts):
        """Free pages for so many tokens of each of several sequences, taken together or not
        at all: lists of pages."""
        need = [-(-n // self.size) for n in counts]
        if sum(need) > len(self.free):
            raise MemoryError("the cache has too few free pages")
        return [[self.free.pop() for _ in range(n)] for n in need]

    def give_back(self, pages):
        """What fresh() gave is not used."""
        self.free += sum(pages, [])[::-1]

    def move(self, seq, pages, tokens: int):
        """The sequence lives in these pages from now on, with its first `tokens` places."""
        self.free += self.owned[seq]
        self.owned[seq], self.lens[seq] = pages, tokens

    def release(self, seq):
        self.free += self.owned.pop(seq, [])
        self.lens.pop(seq, None)
        self.seen.pop(seq, None)

    def table(self, seqs):
        """(page_table, seq_lens) of these sequences on the device."""
        return self.rows([self.owned[s] for s in seqs]), torch.tensor(
            [self.lens[s] for s in seqs], dtype=torch.int32, device=self.device)

    def rows(self, pages):
        """A page table of these lists of pages."""
        width = max(len(p) for p in pages)
        return torch.tensor([p + [0] * (width - len(p)) for p in pages], dtype=torch.int32, device=self.device)


class Rotation(NamedTuple):
    """Norm and rotation of queries and keys (see qk.norm_rotate)."""
    q_weight: torch.Tensor  # fp32 [D]
    k_weight: torch.Tensor
    table: torch.Tensor     # qk.rotation_table
    eps: float = 1e-6
    interleaved: bool = False


class AttentionBlock:
    precision, rotation, weights_of = "if4", None, 0

    def __init__(self, w_qkv: torch.Tensor, w_o: torch.Tensor, heads: int, kv_heads: int,
                 pages: int, page_size: int, window: int = 0, sinks: int = 0, precision: str = "if4",
                 rotation: Rotation = None, weights_of: int = 0):
        """w_qkv [(heads + 2 kv_heads) D, hidden] and w_o [hidden, heads D],
        bf16 on the GPU; quantized once, to `precision` ("if4" or "fp8").  weights_of:
        tokens of a sequence that attention weights are summed for, which evict() goes by
        (0: none, and no evict())."""
        if precision not in ("if4", "fp8"):
            raise ValueError(f"precision must be if4 or fp8, not {precision}")
        if weights_of and window:
            raise ValueError("a window counts places in the cache, which evicted tokens leave")
        self.precision, self.rotation, self.weights_of = precision, rotation, weights_of
        self.mass, self.mass_row = (), {}  # the sums, and which row is whose
        self.heads, self.kv_heads = heads, kv_heads
        self.dim = w_qkv.shape[0] // (heads + 2 * kv_heads)
        self.window, self.sinks = window, sinks
        self.w_qkv, self.w_o = self._weights(w_qkv), self._weights(w_o)
        self.cache = kv_cache.empty(pages, page_size, kv_heads, self.dim, w_qkv.device)
        self.pages = Pages(pages, page_size, w_qkv.device)
        self.exps = dict(k_exp=wl.tensor_scale_exp(K_LIMIT), v_exp=wl.tensor_scale_exp(V_LIMIT))

    def _weights(self, w):
        if self.precision == "fp8":
            return fp8.quantize(w, square=True)
        exp = wl.tensor_scale_exp(float(w.abs().max()))
        return (*if4.quantize(w, exp), exp)

    def _linear(self, x, w, exp, dtype=torch.float32):
        """x W^T with x quantized (IF4: at exponent `exp`, and the result is fp32)."""
        if self.precision == "fp8":
            return fp8.gemm(*fp8.quantize(x), *w, dtype=dtype)
        return if4.gemm(*if4.quantize(x, exp), exp, *w)

    def _project(self, x, exp, positions):
        """q, k and v [tokens, heads, D] of one type, normed and rotated."""
        h, kv, d = self.heads, self.kv_heads, self.dim
        qkv = self._linear(x, self.w_qkv, exp, torch.bfloat16).view(-1, h + 2 * kv, d)
        q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        if self.rotation is not None:
            r = self.rotation
            q, k = qk.norm_rotate(q, k, r.q_weight, r.k_weight, r.table, positions, eps=r.eps,
                                  interleaved=r.interleaved)
        return q, k, v

    def _mass_rows(self, seqs):
        """Rows of the sums (one per sequence that has any) of these sequences, on the device."""
        for s in seqs:
            if s not in self.mass_row:
                free = [i for i in range(len(self.mass)) if i not in self.mass_row.values()]
                if not free:
                    more = torch.zeros(max(8, len(self.mass)), self.kv_heads, self.weights_of, device=self.pages.device)
                    self.mass = torch.cat([self.mass, more]) if len(self.mass) else more
                    free = [len(self.mass) - len(more)]
                self.mass_row[s] = free[0]
        return torch.tensor([self.mass_row[s] for s in seqs], dtype=torch.int32, device=self.pages.device)

    def forward(self, x: torch.Tensor, seqs, counts, x_exp: int = -8, out_exp: int = -8):
        """x [sum(counts), hidden] bf16: counts[i] new tokens of sequence seqs[i],
        one sequence after another.  x_exp, out_exp: exponents that the two
        products' activations are quantized with.  Returns [sum(counts), hidden]
        fp32."""
        if self.weights_of and any(self.pages.lens.get(s, 0) + n > self.weights_of for s, n in zip(seqs, counts)):
            raise ValueError(f"a sequence would have more than the {self.weights_of} tokens that weights are summed for")
        positions = None
        if self.rotation is not None:
            positions = self.pages.positions(seqs, counts)
            if max(positions, default=0) >= len(self.rotation.table):
                raise ValueError(f"position {max(positions)} is past the rotation's table of {len(self.rotation.table)}")
            positions = torch.tensor(positions, dtype=torch.int64, device=x.device)
        q, k, v = self._project(x, x_exp, positions)
        slots = self.pages.extend_all(seqs, counts)
        kv_cache.append(self.cache, k, v, torch.tensor(slots, device=x.device), **self.exps)
        table, lens = self.pages.table(seqs)
        starts = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32,
                              device=x.device)
        q = q.bfloat16()
        sizes = dict(max_q=max(counts), max_len=max(self.pages.lens[s] for s in seqs))
        out = kv_cache.attention(q, self.cache, table, lens, starts, window=self.window, sinks=self.sinks,
                                 **sizes, **self.exps)
        if self.weights_of:
            rows = self._mass_rows(seqs)
            kv_evict.accumulate(self.mass, q, self.cache, table, lens, starts, rows=rows, k_exp=self.exps["k_exp"],
                                **sizes)
        return self._linear(out.view(-1, self.heads * self.dim), self.w_o, out_exp)

    def evict(self, seqs, keep: int, recent: int = 0, sinks: int = 0):
        """Cut the caches of these sequences to `keep` tokens of each kv head: the first
        `sinks`, the latest `recent`, and those with the largest sums of attention weights
        since they came.  Sequences that have no more stay as they are.  What is kept goes to
        other pages: there have to be free ones for `keep` tokens of one sequence, else
        MemoryError and nothing is cut."""
        if not self.weights_of:
            raise ValueError("the block keeps no attention weights (weights_of)")
        seqs = list(seqs)
        if len(set(seqs)) != len(seqs):
            raise ValueError("a sequence comes twice")
        if keep <= 0 or recent < 0 or sinks < 0 or recent + sinks > keep:
            raise ValueError("keep must be positive, recent and sinks not negative, nor more than keep together")
        long = [s for s in seqs if self.pages.lens[s] > keep]
        # as many at once as the free pages allow, whose old pages, which are no fewer, are
        # free for the next ones then
        each = -(-keep // self.pages.size)
        while long:
            some = long[:max(1, len(self.pages.free) // each)]
            self._cut(some, keep, recent, sinks)
            long = long[len(some):]

    def _cut(self, seqs, keep, recent, sinks):
        table, lens = self.pages.table(seqs)
        rows = self._mass_rows(seqs)
        fresh = self.pages.fresh([keep] * len(seqs))
        try:
            new_table = self.pages.rows(fresh)
            kept = kv_evict.select(self.mass, lens, keep, recent=recent, sinks=sinks, rows=rows, mass_out=self.mass)
        except BaseException:  # (no memory for a result or a workspace: nothing has been launched)
            self.pages.give_back(fresh)
            raise
        kv_evict.compact(self.cache, table, kept, new_table)
        for s, pages in zip(seqs, fresh):
            self.pages.move(s, pages, keep)

    def release(self, seq):
        """Forget a sequence: its pages and its sums are free."""
        self.pages.release(seq)
        self.mass_row.pop(seq, None)

    def reference(self, xs, x_exp: int = -8, out_exp: int = -8):
        """The same block on one whole sequence xs [n, hidden], keys and values
        kept as projected, in torch."""
        h, kv, d = self.heads, self.kv_heads, self.dim
        q, k, v = (t.float() for t in self._project(xs, x_exp, torch.arange(len(xs), device=xs.device)))
        k, v = (t.repeat_interleave(h // kv, 1).transpose(0, 1).contiguous() for t in (k, v))
        s = torch.matmul(q.transpose(0, 1).contiguous(), k.transpose(1, 2).contiguous()) * d ** -0.5
        i = torch.arange(len(xs), device=xs.device)
        seen = i <= i[:, None]
        if self.window:
            seen &= (i > i[:, None] - self.window) | (i < self.sinks)
        p = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
        out = torch.matmul(p, v).transpose(0, 1).reshape(-1, h * d)
        return self._linear(out.bfloat16().contiguous(), self.w_o, out_exp)


def random_block(hidden, heads, kv_heads, dim, pages, page_size, window=0, sinks=0, seed=0, rotary=0, positions=0,
                 **kw):
    """A block of random weights; with `rotary` dims rotated, up to `positions` tokens."""
    rows = (heads + 2 * kv_heads) * dim
    w = [torch.from_numpy(wl.normal_weights(*shape, seed + i, std=shape[1] ** -0.5)).bfloat16().cuda()
         for i, shape in enumerate(((rows, hidden), (hidden, heads * dim)))]
    if rotary:
        norm = [torch.from_numpy(1 + wl.normal_weights(1, dim, seed + 2 + i, std=0.1)[0]).float().cuda() for i in range(2)]
        kw["rotation"] = Rotation(*norm, qk.rotation_table(positions, rotary))
    return AttentionBlock(*w, heads, kv_heads, pages, page_size, window, sinks, **kw)


def serve(block, prompts, steps, chunk, hidden, seed=1, keep=0):
    """Prompts of these lengths in chunks, their caches cut to `keep` tokens (0: not), then
    `steps` decode steps of all of them.  Returns (inputs per sequence, outputs per sequence, ms of the prompts, ms
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
    if keep:
        block.evict(range(len(prompts)), keep, recent=keep // 8, sinks=min(4, keep // 8))
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
                        ("window", 0), ("sinks", 0), ("rotary", 0), ("keep", 0)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--precision", choices=("if4", "fp8"), default="if4")
    a = p.parse_args(argv)
    prompts = [max(1, a.prompt - 97 * i) for i in range(a.batch)]
    longest = max(prompts) + a.steps
    pages = sum(-(-(n + a.steps) // a.page_size) for n in prompts) + (a.batch * -(-a.keep // a.page_size))
    block = random_block(a.hidden, a.heads, a.kv_heads, a.dim, pages, a.page_size, a.window, a.sinks, rotary=a.rotary,
                         positions=longest, precision=a.precision, weights_of=longest if a.keep else 0)
    serve(block, [min(64, n) for n in prompts], 1, a.chunk, a.hidden)  # first launches
    for seq in range(a.batch):
        block.release(seq)
    xs, outs, prompt_ms, step_ms = serve(block, prompts, a.steps, a.chunk, a.hidden, keep=a.keep)
    want = block.reference(xs[-1])
    if a.keep:
        outs, want = [o[n:] for o, n in zip(outs, prompts)], want[prompts[-1]:]
    far = float((outs[-1] - want).norm() / want.norm())
    c = block.cache
    used = sum(t.numel() for t in c)
    print(json.dumps({"prompt_tokens": sum(prompts), "prompt_ms": round(prompt_ms, 3),
                      "decode_ms_per_step": round(step_ms, 4), "cache_MB": round(used / 1e6, 1),
                      "bf16_cache_MB": round(4 * c.k_codes.numel() * 2 / 1e6, 1),
                      "rel_error_of_the_if4_cache": round(far, 4)}))


if __name__ == "__main__":
    main()
