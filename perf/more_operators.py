"""Cases of the FP8 block product, of the norm and rotation of queries and keys, and of eviction from the paged IF4 KV cache.

`run` computes each operator in its plain form (elementary torch operations) or, where `own` is true, through
`adaptive_block_scaled_amd`: fp8 (quantize, quantize_t, gemm), qk (norm_rotate, norm_rotate_backward) and kv_evict
(accumulate, select, compact).

FP8 blocks: E4M3 codes and one power of two 2^(byte - 127) per block of 128 values along the contraction dim (a row's blocks,
the last one short where the length is no multiple of 128) or per square of 128 x 128 (weights).  The exponent is the least
e >= -127 with amax * 2^-e <= 448.

The IF4 cache (uint8; `pages` pages of `page_size` tokens, a multiple of 16; groups of 16 along the head dim D):
  k_codes  [pages, kv_heads, page_size, D/2]     k_scales [pages, kv_heads, page_size, D/16]
  v_codes  [pages, kv_heads, page_size/16, 16, 16, D/32]  (tile of 16 tokens, piece of D/16 dims, token, bytes)
  v_scales [pages, kv_heads, page_size/16, D/16, 16]      (tile, group, token)
"""
import math

import torch

own = False

GROUP, BLOCK = 16, 128
DEVICE = "cuda"


# ---------------------------------------------------------------------------------------------------------------------
# Cases

def _linear(name, m, n, k, out="bf16"):
    return dict(name=name, op="linear", m=m, n=n, k=k, out=out)


def _rotate(name, tokens, heads, kv_heads, dim, rotary, dtype, out, interleaved=False):
    return dict(name=name, op="rotate", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rotary=rotary, dtype=dtype, out=out,
                interleaved=interleaved)


def _weights(name, batch, q_lo, q_hi, ctx_lo, ctx_hi, heads, kv_heads, dim, page, window=0, sinks=0):
    return dict(name=name, op="weights", batch=batch, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, window=window, sinks=sinks)


def _evict(name, batch, ctx_lo, ctx_hi, keep, recent, sinks, kv_heads, dim, page):
    return dict(name=name, op="evict", batch=batch, ctx_lo=ctx_lo, ctx_hi=ctx_hi, keep=keep, recent=recent, sinks=sinks,
                kv_heads=kv_heads, dim=dim, page=page)


def listed():
    return [
        # one user's next token through a QKV projection: latency
        _linear("linear_one", 1, 6144, 4096),
        # a serving batch's next tokens through an FFN weight: the weight's bytes
        _linear("linear_batch", 64, 28672, 8192),
        # a prefill or training forward through the same weight
        _linear("linear_ffn", 8192, 28672, 8192),
        # a chunk of odd sizes, a last block of 16 values, fp32 out
        _linear("linear_odd", 1021, 5003, 4112, "f32"),
        # the two backward products of a training layer: three quantizes and two products
        dict(name="linear_grads", op="linear_grads", m=4096, n=4096, k=8192),
        # a decode step's q and k, fp32 columns of the fused projection, to bf16
        _rotate("rotate_decode", 64, 64, 8, 128, 128, "f32", "bf16"),
        # a long prompt's q and k, bf16 columns, half of the dims rotated
        _rotate("rotate_prompt", 8192, 64, 8, 128, 64, "bf16", "bf16"),
        # their gradients in training, with the two weights'
        dict(name="rotate_grads", op="rotate_grads", tokens=4099, heads=32, kv_heads=8, dim=128, rotary=128, dtype="bf16", out="bf16",
             interleaved=False),
        # a decode step's attention weights onto the running sums of a serving batch
        _weights("weights_decode", 64, 1, 1, 3001, 12289, 64, 8, 128, 64),
        # a chunk of a long prompt
        _weights("weights_chunk", 1, 2048, 2048, 16384, 16384, 64, 8, 128, 64),
        # a batch's contexts cut to a quarter, and what is left read back for a check or a move
        _evict("evict_batch", 32, 6001, 8192, 2048, 256, 4, 8, 128, 64),
        # two very long contexts
        _evict("evict_long", 2, 100003, 131071, 32768, 1024, 64, 8, 128, 128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _at_most_listed(case, sizes, step=1):
    """The case with these sizes cut down together until it does no more work than the largest listed one of its operator."""
    tops = [work(c) for c in listed() if c["op"] == case["op"]]
    while any(work(case)[k] > max(t[k] for t in tops) for k in ("bytes", "flops")):
        case.update({n: max(step, case[n] * 4 // 5 // step * step) for n in sizes})
    return case


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grads", "rotate", "rotate_grads", "weights", "weights", "evict"])
    if op == "linear":
        case = _linear("", _log_int(rng, 1, 8192), _log_int(rng, 64, 28672), 16 * _log_int(rng, 4, 512), rng.choice(["bf16", "bf16", "f32"]))
        del case["name"]
        return _at_most_listed(case, ["m"])
    if op == "linear_grads":
        case = dict(op=op, **{s: 16 * _log_int(rng, 4, 512) for s in "mnk"})
        return _at_most_listed(case, ["m", "n", "k"], 16)
    if op in ("rotate", "rotate_grads"):
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 5, 8])
        case = _rotate("", _log_int(rng, 1, 8192), kv * rng.choice([1, 2, 4, 7, 8]), kv, dim, rng.choice([dim, dim, dim // 32 * 16]),
                       rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.3)
        del case["name"]
        case["op"] = op
        return _at_most_listed(case, ["tokens"])
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    kv = rng.choice([1, 2, 4, 5, 8])
    if op == "evict":
        hi = _log_int(rng, 64, 131072)
        keep = max(2, int(hi * rng.uniform(0.05, 1.1)))
        recent = rng.randint(0, keep // 2)
        case = _evict("", _log_int(rng, 1, 64), rng.randint(max(1, hi // 4), hi), hi, keep, recent, min(keep - recent, rng.choice([0, 1, 4, 64])),
                      kv, dim, page)
        del case["name"]
        return _at_most_listed(case, ["batch"])
    kind = rng.choice(["decode", "decode", "chunk", "mixed"])
    if kind == "decode":
        batch, q_lo, q_hi, hi = _log_int(rng, 1, 64), 1, 1, _log_int(rng, 16, 131072)
    elif kind == "chunk":
        batch, q_hi = rng.choice([1, 1, 2, 3]), _log_int(rng, 64, 4096)
        q_lo, hi = rng.randint(max(1, q_hi // 2), q_hi), q_hi + _log_int(rng, 1, 16384)
    else:
        batch, q_lo, q_hi = _log_int(rng, 2, 32), 1, _log_int(rng, 2, 128)
        hi = q_hi + _log_int(rng, 16, 4096)
    window, sinks = (_log_int(rng, 16, 4096), rng.choice([0, 1, 4, 64])) if rng.random() < 0.35 else (0, 0)
    case = _weights("", batch, q_lo, q_hi, rng.randint(max(q_hi, hi // 4), hi), hi, kv * rng.choice([1, 2, 4, 7, 8]), kv, dim, page, window,
                    sinks)
    del case["name"]
    return _at_most_listed(case, ["q_lo", "q_hi", "ctx_lo", "ctx_hi"])


def _spread(lo, hi, n, step):
    """n whole numbers from lo to hi, both included where n > 1, in a mixed order that the case alone decides."""
    return [hi if n == 1 else lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _lengths(case):
    """(new tokens, tokens in the cache) of each sequence."""
    b = case["batch"]
    odd = [s for s in (7, 11, 13) if math.gcd(s, b) == 1][0] if b > 1 else 1
    return _spread(case.get("q_lo", 0), case.get("q_hi", 0), b, 1), _spread(case["ctx_lo"], case["ctx_hi"], b, odd)


def _pairs(case, q_len, ctx):
    """(row, key) pairs that attend, and the keys that any row sees, of one sequence (positions ctx - q_len .. ctx - 1)."""
    pairs, first_seen = 0, ctx - q_len + 1
    for p in range(ctx - q_len, ctx):
        start = max(0, p - case["window"] + 1) if case["window"] else 0
        pairs += p + 1 - start + min(case["sinks"], start)
        first_seen = min(first_seen, start)
    return pairs, ctx - first_seen + min(case["sinks"], first_seen)


def _wide(kind):
    return 4 if kind == "f32" else 2


def work(case):
    op = case["op"]
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k + n * k + m * n * _wide(case["out"]), "flops": 2 * m * n * k}
    if op == "linear_grads":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * n + 2 * m * k + n * k + 2 * m * k + 4 * n * k, "flops": 4 * m * n * k}
    if op in ("rotate", "rotate_grads"):
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        table = case["tokens"] * (8 + 4 * case["rotary"])
        moved = _wide(case["dtype"]) + _wide(case["out"]) + (_wide(case["dtype"]) if op == "rotate_grads" else 0)
        return {"bytes": values * moved + table, "flops": 0}
    d, kvh = case["dim"], case["kv_heads"]
    packed = d // 2 + d // GROUP
    q_lens, ctxs = _lengths(case)
    if op == "evict":
        kept = sum(min(c, case["keep"]) for c in ctxs)
        # the sums in; indices, their sums, and the tokens' K and V out; these in again and read back as bf16
        return {"bytes": kvh * (4 * sum(ctxs) + kept * (8 + 2 * (3 * packed + 2 * d))), "flops": 0}
    seen = [_pairs(case, q, c) for q, c in zip(q_lens, ctxs)]
    keys = sum(k for _, k in seen)
    return {"bytes": 2 * sum(q_lens) * case["heads"] * d + kvh * (packed * keys + 8 * sum(ctxs)),
            "flops": 2 * d * case["heads"] * sum(p for p, _ in seen)}


# ---------------------------------------------------------------------------------------------------------------------
# Inputs

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _vectors(gen, tokens, heads, dim, outliers):
    """Normal values; K has a few channels of a head that are much larger than the others, as trained models have."""
    x = torch.randn(tokens, heads, dim, generator=gen, device=DEVICE)
    if outliers:
        gain = torch.ones(heads, dim, device=DEVICE)
        gain.scatter_(1, torch.randint(0, dim, (heads, max(1, dim // 32)), generator=gen, device=DEVICE), 6.0)
        x *= gain
    return x


def _activations(gen, rows, cols):
    """Normal values with a thousandth of the columns 50 times as large."""
    x = torch.randn(rows, cols, generator=gen, device=DEVICE)
    x[:, torch.randint(0, cols, (max(1, cols // 1000),), generator=gen, device=DEVICE)] *= 50
    return x.bfloat16()


def _gradient(gen, rows, cols):
    """Small values whose size differs from row to row."""
    return (torch.randn(rows, cols, generator=gen, device=DEVICE) * 1e-3
            * torch.exp(torch.randn(rows, 1, generator=gen, device=DEVICE))).bfloat16()


def _weight(gen, rows, cols):
    return torch.randn(rows, cols, generator=gen, device=DEVICE).mul_(cols ** -0.5).bfloat16()


def _exponent(limit):
    """The cache's power of two: set beforehand for values up to `limit`, as a calibration does."""
    return math.ceil(math.log2(limit / (6.0 * 448.0)))


def _if4_rows(x, exp):
    """IF4 codes and scales of x [..., D]: each group in the encoding that is nearer."""
    g = x.float().unflatten(-1, (-1, GROUP))
    a = g.abs()
    sp = (a.amax(-1) * 2.0 ** -exp / 6).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
    u = a / (sp.float() * 2.0 ** exp).unsqueeze(-1)
    half = torch.where(u < 2, 0.5, torch.where(u < 4, 1.0, 2.0))
    c = (torch.round(u / half) * half).clamp(max=6)
    q = torch.round(u * 7 / 6).clamp(max=7)
    pick = (q * 6 / 7 - u).square().sum(-1, keepdim=True) < (c - u).square().sum(-1, keepdim=True)
    index = torch.where(c < 2, 2 * c, torch.where(c < 4, c + 2, c / 2 + 4))
    nib = (torch.where(pick, q, index).to(torch.uint8) + 8 * (g < 0).to(torch.uint8)).flatten(-2)
    return nib[..., 0::2] + 16 * nib[..., 1::2], sp.view(torch.uint8) + 128 * pick.squeeze(-1).to(torch.uint8)


def _filled_cache(gen, pages, page, kv_heads, dim, k_exp, v_exp):
    """A cache that holds K and V of tokens: rows of a pool of quantized tokens, each page's tokens drawn from it."""
    pool = min(4096, pages * page)
    k = _if4_rows(_vectors(gen, pool, kv_heads, dim, True).bfloat16(), k_exp)
    v = _if4_rows(_vectors(gen, pool, kv_heads, dim, False).bfloat16(), v_exp)
    at = torch.randint(0, pool, (pages, page), generator=gen, device=DEVICE)
    kc, ks = (t[at].transpose(1, 2).contiguous() for t in k)
    vc, vs = (t[at].transpose(1, 2) for t in v)
    tiled = (pages, kv_heads, page // 16, 16)
    vc = vc.reshape(*tiled, 16, dim // 32).transpose(3, 4).contiguous()
    vs = vs.reshape(*tiled, dim // GROUP).transpose(3, 4).contiguous()
    return {"k_codes": kc, "k_scales": ks, "v_codes": vc, "v_scales": vs}


def _page_tables(gen, page, *lengths):
    """One page table for each list of lengths, all their pages different, and the number of pages."""
    need = [[-(-n // page) for n in ns] for ns in lengths]
    pages = sum(map(sum, need)) + 5
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    tables, first = [], 0
    for ns in need:
        table = torch.zeros(len(ns), max(ns), dtype=torch.int32, device=DEVICE)
        for b, m in enumerate(ns):
            table[b, :m] = order[first:first + m]
            first += m
        tables.append(table)
    return tables, pages


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op = case["op"]
    state = dict(case=case, op=op)
    if op == "linear":
        state["x"] = _activations(gen, case["m"], case["k"])
        state["w"] = _fp8(_weight(gen, case["n"], case["k"]), True)
        state["out"] = TYPES[case["out"]]
        return state
    if op == "linear_grads":
        state["x"], state["dy"] = _activations(gen, case["m"], case["k"]), _gradient(gen, case["m"], case["n"])
        state["wt"] = _fp8(_weight(gen, case["n"], case["k"]).T.contiguous(), True)
        return state
    if op in ("rotate", "rotate_grads"):
        n, h, kv, d, r = (case[s] for s in ("tokens", "heads", "kv_heads", "dim", "rotary"))
        # q and k as columns of the fused product; each sequence's tokens at consecutive positions, somewhere in its context
        fused = torch.cat([_vectors(gen, n, h, d, True), _vectors(gen, n, kv, d, True), _vectors(gen, n, kv, d, False)], 1)
        fused = fused.to(TYPES[case["dtype"]])
        rows = 40960
        angle = torch.arange(rows, dtype=torch.float64, device=DEVICE)[:, None] * 10000.0 ** (
            -torch.arange(r // 2, dtype=torch.float64, device=DEVICE) * 2 / r)
        first = torch.randint(0, rows - 8192, (max(1, -(-n // 512)),), generator=gen, device=DEVICE).repeat_interleave(512)[:n]
        state.update(
            q=fused[:, :h], k=fused[:, h:h + kv], table=torch.cat([angle.cos(), angle.sin()], 1).float(),
            positions=first + torch.arange(n, device=DEVICE) % 512, out=TYPES[case["out"]], eps=1e-6,
            weights=[1 + 0.2 * torch.randn(d, generator=gen, device=DEVICE) for _ in range(2)])
        if op == "rotate_grads":
            state["dq"], state["dk"] = (_gradient(gen, n * m, d).view(n, m, d).to(state["out"]) for m in (h, kv))
        return state
    kvh, dim, page = case["kv_heads"], case["dim"], case["page"]
    q_lens, ctxs = _lengths(case)
    kept = [min(c, case["keep"]) for c in ctxs] if op == "evict" else []
    tables, pages = _page_tables(gen, page, *([ctxs, kept] if kept else [ctxs]))
    k_exp, v_exp = _exponent(48.0), _exponent(8.0)
    # running sums: what older tokens got so far, very uneven, nothing at all for some of them
    mass = torch.exp(2 * torch.randn(len(ctxs), kvh, max(ctxs), generator=gen, device=DEVICE))
    mass *= torch.rand(mass.shape, generator=gen, device=DEVICE) > 0.1
    state.update(cache=_filled_cache(gen, pages, page, kvh, dim, k_exp, v_exp), k_exp=k_exp, v_exp=v_exp, mass=mass, page_table=tables[0],
                 seq_lens=torch.tensor(ctxs, dtype=torch.int32, device=DEVICE), mass_out=torch.zeros_like(mass), max_len=max(ctxs))
    if op == "evict":
        state["new_table"] = tables[1]
        state["mass_out"] = torch.zeros(len(ctxs), kvh, case["keep"], device=DEVICE)
        # the slots of what is left, sequence by sequence
        at = [(b, torch.arange(n, device=DEVICE)) for b, n in enumerate(kept)]
        state["slots"] = torch.cat([tables[1][b].long()[j // page] * page + j % page for b, j in at])
        state["slot_seq"], state["slot_rank"] = torch.cat([torch.full_like(j, b) for b, j in at]), torch.cat([j for _, j in at])
        return state
    starts = [sum(q_lens[:b]) for b in range(len(q_lens) + 1)]
    state.update(q=_vectors(gen, sum(q_lens), case["heads"], dim, False).bfloat16(), scale=dim ** -0.5, max_q=max(q_lens),
                 q_starts=torch.tensor(starts, dtype=torch.int32, device=DEVICE))
    return state


# ---------------------------------------------------------------------------------------------------------------------
# Plain forms

def _power(e):
    """2^e in fp32, exactly, for whole e from -127 to 127."""
    return torch.where(e == -127, 2.0 ** -127, ((e + 127).int() << 23).view(torch.float32))


def _fp8(x, square=False):
    """E4M3 codes [rows, cols] and the exponent byte of each block, of x [rows, cols], as uint8."""
    rows, cols = x.shape
    tall = BLOCK if square else 1
    padded = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK, 0, -rows % tall))
    g = padded.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, tall))
    a = g.abs().amax((1, 3))
    f, e = torch.frexp(a)
    e = torch.where(f <= 0.875, e - 9, e - 8).clamp(min=-127)  # 448 = 0.875 * 2^9
    zero, bad = a == 0, ~torch.isfinite(a)
    e = torch.where(zero | bad, -127, e)
    codes = (g * _power(-e)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.where(bad[:, None, :, None], 127, codes).flatten(2).flatten(0, 1)[:rows, :cols].contiguous()
    return codes, torch.where(bad, 255, e + 127).to(torch.uint8)


def _fp8_values(codes, scales):
    """fp32 values; scales [rows or ceil(rows / 128), blocks]."""
    rows, cols = codes.shape
    s = torch.where(scales == 255, torch.nan, _power(scales.int() - 127))
    if len(s) != rows:
        s = s.repeat_interleave(BLOCK, 0)[:rows]
    return codes.view(torch.float8_e4m3fn).float().unflatten(0, (rows, 1)).squeeze(1) * s.repeat_interleave(BLOCK, 1)[:, :cols]


def _product(a, w):
    return torch.matmul(_fp8_values(*a), _fp8_values(*w).T)


def _halves(x, rotary, interleaved):
    """The two members of each rotated pair, and the dims that stay."""
    r = x[..., :rotary]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else r.chunk(2, -1)
    return a, b, x[..., rotary:]


def _joined(a, b, rest, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _plain_rotate(state):
    c, s = (t[:, None] for t in state["table"][state["positions"]].chunk(2, -1))
    kind = state["case"]["rotary"], state["case"]["interleaved"]
    outs = []
    for x, w in zip((state["q"], state["k"]), state["weights"]):
        x = x.float()
        z = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + state["eps"]) * w
        a, b, rest = _halves(z, *kind)
        outs.append(_joined(a * c - b * s, a * s + b * c, rest, kind[1]).to(state["out"]))
    return tuple(outs)


def _plain_rotate_grads(state):
    c, s = (t[:, None] for t in state["table"][state["positions"]].chunk(2, -1))
    kind = state["case"]["rotary"], state["case"]["interleaved"]
    dxs, dws = [], []
    for x, w, dy in zip((state["q"], state["k"]), state["weights"], (state["dq"], state["dk"])):
        dtype, x = x.dtype, x.float()
        a, b, rest = _halves(dy.float(), *kind)
        dz = _joined(a * c + b * s, b * c - a * s, rest, kind[1])
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + state["eps"])
        n = x * r
        g = dz * w
        dxs.append((r * (g - n * (g * n).mean(-1, keepdim=True))).to(dtype))
        dws.append((dz * n).sum((0, 1)))
    return (*dxs, *dws)


def _if4_values(codes, scales, exp):
    """fp32 values of IF4 rows: codes [..., D/2], scales [..., D/16]."""
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (-1, GROUP))
    m = (nib & 7).float()
    fp4 = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    sp = (scales & 127).view(torch.float8_e4m3fn).float().unsqueeze(-1)
    y = torch.where((scales >= 128).unsqueeze(-1), 6 * m * sp / 7, fp4 * sp) * 2.0 ** exp
    return torch.where(nib >= 8, -y, y).flatten(-2)


def _plain_weights(state):
    q, c, starts, lens = state["q"], state["cache"], state["q_starts"].long(), state["seq_lens"].long()
    n, kvh = state["max_len"], c["k_codes"].shape[1]
    total, heads, _ = q.shape
    window, sinks = state["case"]["window"], state["case"]["sinks"]
    j = torch.arange(n, device=q.device)
    dense = [c[name][state["page_table"].long()].transpose(1, 2).flatten(2, 3)[:, :, :n] for name in ("k_codes", "k_scales")]
    k = _if4_values(*dense, state["k_exp"])  # [batch, kv_heads, n, D]
    rows_of = starts[1:] - starts[:-1]
    out = state["mass_out"]
    new = j >= (lens - rows_of)[:, None]
    out.copy_(torch.where(j < lens[:, None], torch.where(new, 0, state["mass"].transpose(0, 1)), out.transpose(0, 1)).transpose(0, 1))
    i = torch.arange(state["max_q"], device=q.device)
    step = max(1, 2 ** 29 // (len(lens) * heads * n))  # as many rows at a time as 2 GB of scores hold
    for r in range(0, state["max_q"], step):
        i = torch.arange(r, min(r + step, state["max_q"]), device=q.device)
        there = i < rows_of[:, None]
        x = q.float()[(starts[:-1, None] + i).clamp(max=total - 1)].unflatten(2, (kvh, -1)).permute(0, 2, 3, 1, 4)
        s = torch.matmul(x.flatten(2, 3), k.transpose(2, 3).contiguous()).mul_(state["scale"]).unflatten(2, (-1, len(i)))
        pos = (lens - rows_of)[:, None, None] + i[:, None]
        seen = (j <= pos) & there[:, :, None]
        if window:
            seen &= (j > pos - window) | (j < sinks)
        s = s.masked_fill_(~seen[:, None, None], -torch.inf)
        e = s.sub_(s.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
        e /= e.sum(-1, keepdim=True).clamp(min=1e-30)
        out += torch.where((j < lens[:, None])[:, None], e.sum((2, 3)), 0)
    return out


def _plain_evict(state):
    case, mass, lens = state["case"], state["mass"], state["seq_lens"].long()
    keep, page, c = case["keep"], case["page"], state["cache"]
    j = torch.arange(mass.shape[2], device=mass.device)
    at = j[None, None]
    n = lens[:, None, None]
    always = (at < case["sinks"]) | (at >= n - case["recent"])
    order = torch.where(at >= n, -torch.inf, torch.where(always, torch.inf, mass))
    top = torch.sort(order, dim=-1, descending=True, stable=True)[1][..., :keep]
    if top.shape[-1] < keep:
        top = torch.nn.functional.pad(top, (0, keep - top.shape[-1]), value=mass.shape[2])
    top = torch.where(torch.arange(keep, device=mass.device) < lens.clamp(max=keep)[:, None, None], top, 1 << 40).sort(-1)[0]
    there = top < 1 << 40
    kept = torch.where(there, top, -1).int()
    safe = torch.where(there, top, 0)
    out = state["mass_out"]
    out.copy_(torch.where(there, mass.gather(2, safe), out))
    # tokens as rows of the cache, moved into the new pages and read back from there
    vc, vs = (c[name].transpose(3, 4) for name in ("v_codes", "v_scales"))
    vc, vs = vc.flatten(4).flatten(2, 3), vs.flatten(2, 3)
    b, r = state["slot_seq"], state["slot_rank"]
    token = safe[b, :, r]  # [slots, kv_heads]
    p, o = state["page_table"].long()[b[:, None], token // page], token % page
    h = torch.arange(token.shape[1], device=token.device)
    new_p, new_o = state["slots"] // page, state["slots"] % page
    rows = [t[p, h, o] for t in (c["k_codes"], c["k_scales"], vc, vs)]
    c["k_codes"][new_p, :, new_o], c["k_scales"][new_p, :, new_o] = rows[:2]
    c["v_codes"][new_p, :, new_o // 16, :, new_o % 16] = rows[2].unflatten(-1, (16, -1))
    c["v_scales"][new_p, :, new_o // 16, :, new_o % 16] = rows[3]
    return (kept, out, _if4_values(*rows[:2], state["k_exp"]).bfloat16(), _if4_values(*rows[2:], state["v_exp"]).bfloat16())


def run(state):
    op = state["op"]
    if own:
        from adaptive_block_scaled_amd import fp8, kv_cache, kv_evict, qk
        if op == "linear":
            return fp8.gemm(*fp8.quantize(state["x"]), *state["w"], dtype=state["out"])
        if op == "linear_grads":
            dx = fp8.gemm(*fp8.quantize(state["dy"]), *state["wt"], dtype=torch.bfloat16)
            dw = fp8.gemm(*fp8.quantize_t(state["dy"]), *fp8.quantize_t(state["x"]), dtype=torch.float32)
            return dx, dw
        if op == "rotate":
            return qk.norm_rotate(state["q"], state["k"], *state["weights"], state["table"], state["positions"], eps=state["eps"],
                                  interleaved=state["case"]["interleaved"], dtype=state["out"])
        if op == "rotate_grads":
            return qk.norm_rotate_backward(state["dq"], state["dk"], state["q"], state["k"], *state["weights"], state["table"],
                                           state["positions"], eps=state["eps"], interleaved=state["case"]["interleaved"])
        cache = kv_cache.KVCache(**state["cache"])
        if op == "weights":
            return kv_evict.accumulate(state["mass"], state["q"], cache, state["page_table"], state["seq_lens"], state["q_starts"],
                                       max_q=state["max_q"], max_len=state["max_len"], scale=state["scale"], k_exp=state["k_exp"],
                                       window=state["case"]["window"], sinks=state["case"]["sinks"], out=state["mass_out"])
        kept = kv_evict.select(state["mass"], state["seq_lens"], state["case"]["keep"], recent=state["case"]["recent"],
                               sinks=state["case"]["sinks"], mass_out=state["mass_out"])
        kv_evict.compact(cache, state["page_table"], kept, state["new_table"])
        return (kept, state["mass_out"], *kv_cache.read(cache, state["slots"], k_exp=state["k_exp"], v_exp=state["v_exp"]))
    if op == "linear":
        return _product(_fp8(state["x"]), state["w"]).to(state["out"])
    if op == "linear_grads":
        dy, x = state["dy"], state["x"]
        return _product(_fp8(dy), state["wt"]).bfloat16(), _product(_fp8(dy.T), _fp8(x.T))
    return {"rotate": _plain_rotate, "rotate_grads": _plain_rotate_grads, "weights": _plain_weights, "evict": _plain_evict}[op](state)


# ---------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits

_E4M3 = [m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]
_FP4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_INT4 = [6 * i / 7 for i in range(8)]


def _two_to(e):
    """2^e in 64 bits, exactly (whole e as 64-bit numbers)."""
    return ((e + 1023).long() << 52).view(torch.float64)


def _exact_fp8(x):
    """What x [rows, cols] is after its rows' blocks have been encoded."""
    grid = torch.tensor(_E4M3, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[1], BLOCK):
        v = x[:, c:c + BLOCK].double()
        top = v.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(top / 448)).nan_to_num(neginf=-127)
        e = torch.where(top > 448 * _two_to(e), e + 1, torch.where(top <= 448 * _two_to(e - 1), e - 1, e)).clamp(min=-127)
        u = v.abs() / _two_to(e)
        up, down = torch.bucketize(u, mid, right=True), torch.bucketize(u, mid)
        out[:, c:c + BLOCK] = grid[torch.where(up % 2 == 0, up, down)] * _two_to(e) * torch.sign(v)
    return out


def _exact_codes(codes, scales):
    """64-bit values of FP8 codes with square blocks."""
    table = torch.tensor(_E4M3 + [math.nan], dtype=torch.float64, device=codes.device)
    table = torch.cat([table, -table])
    s = _two_to(scales.double() - 127)
    out = torch.empty(codes.shape, dtype=torch.float64, device=codes.device)
    for r in range(len(s)):
        rows = codes[r * BLOCK:(r + 1) * BLOCK]
        out[r * BLOCK:(r + 1) * BLOCK] = table[rows.long()] * s[r].repeat_interleave(BLOCK)[:codes.shape[1]]
    return out


def _exact_rows(codes, scales, exp):
    """64-bit values of IF4 rows, by tables of every byte."""
    table = torch.tensor(_E4M3 + [math.nan], dtype=torch.float64, device=codes.device)
    both = torch.tensor([_FP4 + [-v for v in _FP4], _INT4 + [-v for v in _INT4]], dtype=torch.float64, device=codes.device)
    kind, s = (scales.long() >> 7).repeat_interleave(GROUP, -1), table[scales.long() & 127].repeat_interleave(GROUP, -1)
    nib = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.long, device=codes.device)
    nib[..., 0::2], nib[..., 1::2] = codes & 15, codes >> 4
    return both[kind, nib] * s * 2.0 ** exp


def _exact_rotation(state):
    """Cosine and sine of every token and pair, as a complex number [tokens, 1, R/2] (the table's own values)."""
    r = state["case"]["rotary"] // 2
    t = state["table"][state["positions"]].double()
    return torch.complex(t[:, :r], t[:, r:])[:, None]


def _exact_turn(z, turn, rotary, interleaved):
    """z with its pairs, as complex numbers, multiplied by `turn`."""
    out = z.clone()
    half = rotary // 2
    first = (2 if interleaved else 1) * torch.arange(half, device=z.device)
    second = first + (1 if interleaved else half)
    p = torch.complex(z[..., first], z[..., second]) * turn
    out[..., first], out[..., second] = p.real, p.imag
    return out


def _exact_rotate(state, grads):
    turn, kind = _exact_rotation(state), (state["case"]["rotary"], state["case"]["interleaved"])
    outs, dws = [], []
    for i, name in enumerate("qk"):
        x, w = state[name].double(), state["weights"][i].double()
        size = (x.square().sum(-1, keepdim=True) / x.shape[-1] + state["eps"]).sqrt()
        if not grads:
            outs.append(_exact_turn(x / size * w, turn, *kind))
            continue
        dz = _exact_turn(state["d" + name].double(), turn.conj(), *kind)
        g = dz * w
        outs.append(g / size - x * (g * x).sum(-1, keepdim=True) / (x.shape[-1] * size ** 3))
        dws.append((dz * x / size).flatten(0, 1).sum(0))
    return (*outs, *dws)


def _exact_weights(case, state):
    if work(case)["flops"] > 2e12:
        return None
    c, page, kvh = state["cache"], case["page"], case["kv_heads"]
    out = state["mass_out"].double()
    group = case["heads"] // kvh
    first = 0
    for b, (q_len, ctx) in enumerate(zip(*_lengths(case))):
        key = torch.arange(ctx, device=DEVICE)
        p, o = state["page_table"][b].long()[key // page], key % page
        old = ctx - q_len
        out[b, :, :old], out[b, :, old:ctx] = state["mass"][b, :, :old].double(), 0
        for h in range(kvh):
            k = _exact_rows(c["k_codes"][p, h, o], c["k_scales"][p, h, o], state["k_exp"])
            for r in range(0, q_len, 512):
                n = min(512, q_len - r)
                pos = old + r + torch.arange(n, device=DEVICE)[:, None]
                hidden = key > pos
                if case["window"]:
                    hidden |= (key <= pos - case["window"]) & (key >= case["sinks"])
                for m in range(h * group, (h + 1) * group):
                    s = (state["q"][first + r:first + r + n, m].double() @ k.T) * state["scale"]
                    out[b, h, :ctx] += torch.softmax(s.masked_fill(hidden, -math.inf), -1).sum(0)
        first += q_len
    return out


def _exact_evict(case, state):
    c, page, kvh, keep = state["cache"], case["page"], case["kv_heads"], case["keep"]
    kept = torch.full((case["batch"], kvh, keep), -1, dtype=torch.int32, device=DEVICE)
    mass = state["mass_out"].double()
    ks, vs = [], []
    for b, ctx in enumerate(_lengths(case)[1]):
        n = min(ctx, keep)
        last = max(ctx - case["recent"], 0)
        first = min(case["sinks"], last)
        rows = []
        for h in range(kvh):
            if ctx <= keep:
                at = torch.arange(ctx, device=DEVICE)
            else:
                some = state["mass"][b, h, first:last].double()
                want = keep - first - (ctx - last)
                order = (-some).argsort(stable=True)[:want]
                at = torch.cat([torch.arange(first, device=DEVICE), order.sort()[0] + first, torch.arange(last, ctx, device=DEVICE)])
            kept[b, h, :n], mass[b, h, :n] = at.int(), state["mass"][b, h, at].double()
            p, o = state["page_table"][b].long()[at // page], at % page
            rows.append((_exact_rows(c["k_codes"][p, h, o], c["k_scales"][p, h, o], state["k_exp"]),
                         _exact_rows(c["v_codes"][p, h, o // 16, :, o % 16].reshape(n, -1), c["v_scales"][p, h, o // 16, :, o % 16],
                                     state["v_exp"])))
        ks.append(torch.stack([k for k, _ in rows], 1))
        vs.append(torch.stack([v for _, v in rows], 1))
    return kept, mass, torch.cat(ks), torch.cat(vs)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _exact_fp8(state["x"]) @ _exact_codes(*state["w"]).T
    if op == "linear_grads":
        return (_exact_fp8(state["dy"]) @ _exact_codes(*state["wt"]).T,
                _exact_fp8(state["dy"].T.contiguous()) @ _exact_fp8(state["x"].T.contiguous()).T)
    if op in ("rotate", "rotate_grads"):
        return _exact_rotate(state, op == "rotate_grads")
    return _exact_weights(case, state) if op == "weights" else _exact_evict(case, state)
