"""Norm and rotation of queries and keys, and its gradients, against the formulas in 64 bits,
element by element, within bounds that follow from fp32 arithmetic; the gradients also
against differences."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}  # half a step of a type, relative to the value


@pytest.fixture(scope="module")
def qk():
    from adaptive_block_scaled_amd import qk
    return qk


def turned(z, cos, sin, rotary, interleaved, sign=1.0):
    """z [..., D] with its pairs turned by sign * angle."""
    out = z.clone()
    i = torch.arange(rotary // 2)
    x, y = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    out[..., x] = z[..., x] * cos - sign * z[..., y] * sin
    out[..., y] = sign * z[..., x] * sin + z[..., y] * cos
    return out


def larger(z, cos, sin, rotary, interleaved):
    """|a| |cos| + |b| |sin|: what the two products of a turned value amount to."""
    return turned(z.abs(), cos.abs(), -sin.abs(), rotary, interleaved).abs().maximum(
        turned(z.abs(), cos.abs(), sin.abs(), rotary, interleaved).abs())


def angles(table, positions, rotary):
    t = table.double().cpu()[positions.cpu()][:, None]
    return t[..., :rotary // 2], t[..., rotary // 2:]


def forward(x, w, table, positions, eps, rotary, interleaved):
    """(y, bound): a norm of D squares is off by no more than D/2 + 4 roundings, a turned
    value by three more of its two products."""
    x, w = x.double().cpu(), w.double().cpu()
    cos, sin = angles(table, positions, rotary)
    z = x * (x.square().mean(-1, keepdim=True) + eps) ** -0.5 * w
    bound = larger(z, cos, sin, rotary, interleaved) * (x.shape[-1] / 2 + 16) * 2.0 ** -24
    return turned(z, cos, sin, rotary, interleaved), bound


def backward(x, w, dy, table, positions, eps, rotary, interleaved):
    """(dx, dw, their bounds)"""
    x, w, dy = (t.double().cpu() for t in (x, w, dy))
    cos, sin = angles(table, positions, rotary)
    dz = turned(dy, cos, sin, rotary, interleaved, -1.0)
    r = (x.square().mean(-1, keepdim=True) + eps) ** -0.5
    g, gm = dz * w, larger(dy, cos, sin, rotary, interleaved)
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    d = x.shape[-1]
    bx = r * (gm * w.abs() + x.abs() * r * r * (gm * w.abs() * x.abs()).mean(-1, keepdim=True)) * (2 * d + 32) * 2.0 ** -24
    bw = (gm * x.abs() * r).sum((0, 1)) * (x.shape[0] * x.shape[1] + d + 16) * 2.0 ** -24
    return dx, (dz * x * r).sum((0, 1)), bx, bw


def near(got, want, bound):
    got = got.double().cpu()
    assert got.shape == want.shape
    tol = bound + (want.abs() + bound) * STEP.get(got.dtype, 0)
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() - tol).max())


def inputs(tokens, heads, kv_heads, dim, rotary, dtype, out_dtype, seed=0, rows=5000):
    g = torch.Generator().manual_seed(seed)
    fused = torch.randn(tokens, heads + 2 * kv_heads, dim, generator=g) * torch.exp(
        torch.randn(tokens, heads + 2 * kv_heads, 1, generator=g))
    fused = fused.to(dtype).cuda()
    w = [(1 + 0.3 * torch.randn(dim, generator=g)).cuda() for _ in range(2)]
    from adaptive_block_scaled_amd import qk
    table = qk.rotation_table(rows, rotary) if rotary else torch.zeros(rows, 0, device="cuda")
    pos = torch.randint(0, rows, (tokens,), generator=g).cuda()
    dy = [(torch.randn(tokens, h, dim, generator=g) * 0.1).to(out_dtype).cuda() for h in (heads, kv_heads)]
    return fused[:, :heads], fused[:, heads:heads + kv_heads], w, table, pos, dy


def rounded(bound, want, dtype):
    return bound + (want.abs() + bound) * STEP[dtype]


# every lane count, dims that leave lanes empty, part of the dims turned, none, one token and many
SHAPES = [(1, 1, 1, 64, 64), (3, 4, 2, 128, 128), (5, 6, 3, 256, 256), (17, 7, 1, 80, 32), (9, 5, 5, 96, 96),
          (33, 32, 8, 128, 64), (2, 3, 1, 8, 8), (4, 2, 2, 72, 24), (4, 2, 2, 72, 48), (2, 3, 1, 16, 16), (3, 2, 1, 176, 112), (6, 8, 4, 128, 0), (700, 16, 4, 64, 64)]
# (pairs of two halves: rotary is a multiple of 16)
KINDS = [(*s, il) for s in SHAPES for il in (False, True) if il or s[4] % 16 == 0]
TYPES = [(BF16, BF16), (F32, BF16), (F32, F32), (BF16, F32)]


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("tokens,heads,kv,dim,rotary,interleaved", KINDS)
def test_forward(qk, tokens, heads, kv, dim, rotary, dtype, out, interleaved):
    q, k, w, table, pos, _ = inputs(tokens, heads, kv, dim, rotary, dtype, out)
    got = qk.norm_rotate(q, k, *w, table, pos, eps=1e-5, interleaved=interleaved, dtype=out)
    for y, x, wt in zip(got, (q, k), w):
        assert y.dtype == out
        want, bound = forward(x, wt, table, pos, 1e-5, rotary, interleaved)
        near(y.double(), want, rounded(bound, want, out))


@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("tokens,heads,kv,dim,rotary,interleaved", KINDS)
def test_backward(qk, tokens, heads, kv, dim, rotary, dtype, out, interleaved):
    q, k, w, table, pos, dy = inputs(tokens, heads, kv, dim, rotary, dtype, out, 1)
    got = qk.norm_rotate_backward(*dy, q, k, *w, table, pos, eps=1e-5, interleaved=interleaved)
    for i, (x, wt, d) in enumerate(zip((q, k), w, dy)):
        assert got[i].dtype == dtype and got[2 + i].dtype == F32
        dx, dw, bx, bw = backward(x, wt, d, table, pos, 1e-5, rotary, interleaved)
        near(got[i].double(), dx, rounded(bx, dx, dtype))
        near(got[2 + i].double(), dw, rounded(bw, dw, F32))


def test_gradients_against_differences(qk):
    """<dy, y> as a function of one value at a time, by central differences in 64 bits."""
    q, k, w, table, pos, dy = inputs(2, 2, 1, 24, 16, F32, F32, 2)
    got = qk.norm_rotate_backward(*dy, q, k, *w, table, pos, eps=1e-3)

    def value(x, wt, d):
        return float((forward(x, wt, table, pos, 1e-3, 16, False)[0] * d.double().cpu()).sum())
    for i, (x, wt, d) in enumerate(zip((q, k), w, dy)):
        x, wt = x.double().cpu(), wt.double().cpu()
        for of, grad in ((x, got[i]), (wt, got[2 + i])):
            flat = of.reshape(-1)  # x: a copy, and put back below
            for e in range(0, flat.numel(), 3):
                lo, hi = flat.clone(), flat.clone()
                lo[e] -= 1e-4
                hi[e] += 1e-4
                a, b = (value(t.view_as(of), wt, d) if of is x else value(x, t, d) for t in (hi, lo))
                # truncation ~ 1e-8 of the third derivative, rounding 1e-16 / 1e-4
                assert abs((a - b) / 2e-4 - float(grad.reshape(-1)[e])) <= 1e-5


@pytest.mark.parametrize("tokens,heads,kv", [(8192, 16, 2), (1, 64, 8), (513, 1, 1)])
def test_many_vectors(qk, tokens, heads, kv):
    # long runs of heads per wave, and sums over many workgroups
    q, k, w, table, pos, dy = inputs(tokens, heads, kv, 128, 128, BF16, BF16, 3)
    got = qk.norm_rotate(q, k, *w, table, pos)
    grads = qk.norm_rotate_backward(*dy, q, k, *w, table, pos)
    for i, (x, wt, d) in enumerate(zip((q, k), w, dy)):
        want, bound = forward(x, wt, table, pos, 1e-6, 128, False)
        near(got[i].double(), want, rounded(bound, want, BF16))
        dx, dw, bx, bw = backward(x, wt, d, table, pos, 1e-6, 128, False)
        near(grads[i].double(), dx, rounded(bx, dx, BF16))
        near(grads[2 + i].double(), dw, rounded(bw, dw, F32))
    assert torch.equal(grads[2], qk.norm_rotate_backward(*dy, q, k, *w, table, pos)[2])


def test_in_place_and_strides(qk):
    q, k, w, table, pos, dy = inputs(21, 6, 2, 128, 64, BF16, BF16, 4)
    want = qk.norm_rotate(q, k, *w, table, pos)
    q2, k2 = q.clone(), k.clone()
    assert qk.norm_rotate(q2, k2, *w, table, pos, out=(q2, k2))[0] is q2
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    # heads before tokens, and outputs as parts of wider buffers that keep the rest
    qt, kt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k))
    back = torch.full((21, 11, 128), 7.0, dtype=BF16, device="cuda")
    got = qk.norm_rotate(qt, kt, *w, table, pos, out=(back[:, 1:7], back[:, 8:10]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((back[:, [0, 7, 10]] == 7.0).all())
    grads = qk.norm_rotate_backward(*dy, q, k, *w, table, pos)
    dq, dk = dy[0].clone(), dy[1].clone()
    qk.norm_rotate_backward(dq, dk, q, k, *w, table, pos, out=(dq, dk))
    assert torch.equal(dq, grads[0]) and torch.equal(dk, grads[1])


def test_skipped_tokens(qk):
    q, k, w, table, pos, dy = inputs(40, 5, 1, 64, 64, F32, F32, 5, rows=100)
    want = qk.norm_rotate(q, k, *w, table, pos)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[0, 7, 8, 39]] = True
    at = pos.clone()
    at[bad] = torch.tensor([-1, 100, 1 << 40, -(1 << 62)], device="cuda")
    out = tuple(torch.full_like(t, 7.0).contiguous() for t in want)
    qk.norm_rotate(q, k, *w, table, at, out=out)
    for y, z in zip(out, want):
        assert bool((y[bad] == 7.0).all()) and torch.equal(y[~bad], z[~bad])
    grads = qk.norm_rotate_backward(*dy, q, k, *w, table, at)
    only = qk.norm_rotate_backward(*(d[~bad].contiguous() for d in dy), q[~bad], k[~bad], *w, table, pos[~bad])
    for i in range(2):
        assert not bool(grads[i][bad].any()) and torch.equal(grads[i][~bad], only[i])
        assert float((grads[2 + i] - only[2 + i]).norm()) <= 1e-5 * float(only[2 + i].norm())


def test_zero_vectors_and_values_of_no_use(qk):
    q, k, w, table, pos, dy = inputs(6, 4, 2, 96, 96, BF16, BF16, 6)
    q, k = q.clone(), k.clone()
    q[2, 1] = 0
    k[3, 0, 5] = float("nan")
    y = qk.norm_rotate(q, k, *w, table, pos)
    assert not bool(y[0][2, 1].any()) and not bool(y[0].isnan().any())
    assert bool(y[1][3, 0].isnan().all()) and int(y[1].isnan().sum()) == 96
    dx = qk.norm_rotate_backward(*dy, q, k, *w, table, pos)
    assert bool(dx[0].isfinite().all()) and int(dx[1].isnan().sum()) == 96


def test_nothing(qk):
    q, k, w, table, pos, dy = inputs(4, 3, 2, 64, 64, BF16, BF16, 7)
    assert qk.norm_rotate(q[:0], k[:0], *w, table, pos[:0])[0].shape == (0, 3, 64)
    grads = qk.norm_rotate_backward(dy[0][:0], dy[1][:0], q[:0], k[:0], *w, table, pos[:0])
    assert not bool(grads[2].any()) and not bool(grads[3].any())
    none = k[:, :0]
    y = qk.norm_rotate(q, none, *w, table, pos)
    assert torch.equal(y[0], qk.norm_rotate(q, k, *w, table, pos)[0]) and y[1].shape == (4, 0, 64)
    grads = qk.norm_rotate_backward(dy[0], dy[1][:, :0], q, none, *w, table, pos)
    assert torch.equal(grads[2], qk.norm_rotate_backward(*dy, q, k, *w, table, pos)[2]) and not bool(grads[3].any())


def test_far_positions(qk):
    # the table's angles are right where 32 bits would be off by 0.03
    table = qk.rotation_table(1 << 20, 64)
    p = (1 << 20) - 1
    want = np.cos(p * 10000.0 ** (-2 * np.arange(32) / 64))
    assert np.abs(table[p, :32].cpu().numpy() - want).max() <= 2.0 ** -24


def test_other_stream_and_graph(qk):
    q, k, w, table, pos, dy = inputs(30, 8, 2, 128, 128, BF16, BF16, 8)
    q, k = q.contiguous(), k.contiguous()

    def step():
        y = qk.norm_rotate(q, k, *w, table, pos)
        return (*y, *qk.norm_rotate_backward(*dy, q, k, *w, table, pos))
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        q.mul_(1.5), k.mul_(-1), pos.copy_(pos.flip(0))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_refusals(qk):
    q, k, w, table, pos, dy = inputs(4, 4, 2, 64, 64, BF16, BF16, 9)
    ok = dict(q=q, k=k, q_weight=w[0], k_weight=w[1], table=table, positions=pos)
    bad = [dict(q=q.half()), dict(q=q.cpu()), dict(k=k.float()), dict(k=k[:3]), dict(k=k[..., :32]), dict(q=q[0]),
           dict(q_weight=w[0].bfloat16()), dict(k_weight=w[1][:32]), dict(table=table[:, :60]), dict(table=table[:, :24].contiguous()), dict(table=table[:, ::2]),
           dict(table=table.double()), dict(positions=pos.int()), dict(positions=pos[:3]), dict(eps=-1.0),
           dict(eps=float("nan")), dict(dtype=torch.float16), dict(out=(q.float(), k)), dict(q=q.transpose(1, 2)),
           dict(out=(q[:, :1].expand(4, 4, 64), k)), dict(table=qk.rotation_table(10, 128))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            qk.norm_rotate(**{**ok, **kw})
    wide = torch.zeros(4, 4, 264, dtype=BF16, device="cuda")
    for x in (wide, wide[..., :60], wide[..., 4:68]):
        with pytest.raises((ValueError, RuntimeError)):
            qk.norm_rotate(x, x, torch.ones(x.shape[2], device="cuda"), torch.ones(x.shape[2], device="cuda"), table, pos)
    for d in ((dy[0].float(), dy[1]), (dy[0][:3], dy[1]), (dy[0], dy[1].cpu()), (None, dy[1])):
        with pytest.raises(ValueError):
            qk.norm_rotate_backward(*d, **ok)
    with pytest.raises(ValueError, match="workspace"):
        qk.norm_rotate_backward(*dy, **ok, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="rotary"):
        qk.rotation_table(10, 12)
