"""Plain float64 forms of the expert layer's operators, with bounds on how far
a float32 computation of the same formula may be from them.

Half a rounding step relative to the value is 2^-8 for bf16, 2^-4 for e4m3
(and half its smallest step, 2^-10 of the scale, below its normal range) and
2^-24 for float32.  A sum of n terms in float32, in any order, is off by at
most (n - 1) * u * sum |terms| with u = 2^-24 if every addition rounds to
nearest and 2^-23 if it truncates; matrix instructions are given the latter
for the 128 (or, with the split activation, 256) terms of a block.
"""
from __future__ import annotations

import torch

F8 = torch.float8_e4m3fn
U = 2.0 ** -24
BF16_HALF, E4M3_HALF, E4M3_SUB = 2.0 ** -8, 2.0 ** -4, 2.0 ** -10


def values(q, s, per=1):
    """float64 values of e4m3 bytes [R, C] with scales [ceil(R/per), C/128]."""
    v = q.view(F8).double()
    return v * s.double().repeat_interleave(per, 0)[:v.shape[0]].repeat_interleave(128, 1)


def quantise(v):
    """e4m3 bytes and scales (amax / 448) of float32 rows [R, C]."""
    b = v.float().reshape(v.shape[0], -1, 128)
    s = b.abs().amax(-1) / 448.0
    q = torch.where(s[..., None] > 0, b / s[..., None], torch.zeros_like(b)).to(F8)
    return q.view(torch.uint8).reshape(v.shape), s


def weights(E, out, cols, gen, device="cuda", std=None):
    """Random block-scaled e4m3 weights [E, out, cols], scales [E, ceil(out/128), cols/128]."""
    nb, kb = -(-out // 128), cols // 128
    w = torch.randn((E, nb, 128, kb, 128), generator=gen, device=device) * (cols ** -0.5 if std is None else std)
    s = w.abs().amax((2, 4)) / 448.0
    q = (w / s[:, :, None, :, None]).to(F8).view(torch.uint8)
    return q.reshape(E, nb * 128, cols)[:, :out].contiguous(), s.contiguous()


def sum_bound(K, terms_per_block=128, joins=8):
    """Relative to sum |terms|: the blocks' own sums, then one fused
    multiply-add a block, and `joins` further roundings."""
    return (terms_per_block + 2) * 2 * U + (K // 128 + joins) * U


def product(xv, wv, K, **kw):
    """y = x w^T and its bound."""
    return xv @ wv.T, (xv.abs() @ wv.abs().T) * sum_bound(K, **kw)


def silu_mul(g, dg, u, du):
    """silu(g) * u and its bound from those of g and u: |silu'| <= 1.1; the
    exponential's argument is rounded (|g| * 2^-23, at most 2^-16 where the
    exponential is not negligible against 1) and a handful of roundings follow."""
    s = g / (1 + torch.exp(-g))
    a = s * u
    rel = (torch.clamp(g.abs(), max=110.0) * 2 + 12) * U
    return a, 1.1 * dg * (u.abs() + du) + s.abs() * du + a.abs() * rel


def check_quantised(q, s, v, dv, what=""):
    """8-bit rows against float64 values v with bound dv."""
    R, C = v.shape
    b, db = v.reshape(R, -1, 128), dv.reshape(R, -1, 128)
    amax, near = b.abs().amax(-1), db.amax(-1)
    s = s.double()
    off = (s - amax / 448.0).abs()
    assert bool((off <= near / 448.0 + 4 * U * amax / 448.0 + 1e-44).all()), f"{what} scale off by {off.max().item()}"
    got = q.view(F8).double().reshape(R, -1, 128) * s[..., None]
    lim = E4M3_HALF * (b.abs() + db) + E4M3_SUB * 1.01 * s[..., None] + 3 * db + 1e-44
    bad = (got - b).abs() > lim
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} bytes off, worst {((got - b).abs() / lim).max().item()}"


def check_bf16(got, ref, bound, what=""):
    lim = BF16_HALF * (ref.abs() + bound) + bound + 2.0 ** -133
    d = (got.double() - ref).abs()
    bad = ~(d <= lim)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {(d / lim).max().item()}"
    # over many values an error is spread over the half step: 2^-8 / sqrt(3) of the norm at the most
    if ref.numel() >= 4096:
        rel = (d.norm() / ref.norm()).item()
        assert rel <= BF16_HALF / 3 ** 0.5 * 1.01, f"{what}: {rel} of the norm"


def group_rows(exp_off, rows, R):
    """[(expert, first row, rows)] of the expert-major layout."""
    eo = exp_off.cpu().tolist()
    out, base, e = [], 0, 0
    for d, off in enumerate(eo):
        start = d * R if R else base
        cap = R if R else rows
        for a, b in zip(off, off[1:]):
            a, b = min(a, cap), min(b, cap)
            out.append((e, start + a, b - a))
            e += 1
        base += off[-1]
    return out


def _e4m3_products(xv, wv):
    """What an e4m3 matrix instruction may lose against exact products: it adds
    eight products (of consecutive columns) at a time on a grid of 2^-13 of the
    power of two of the largest one, towards zero.  The largest loses nothing
    (a product of two 4-bit significands has 6 bits behind the point), the
    other seven less than 2^-13 of it each."""
    most = lambda v: v.abs().reshape(v.shape[0], -1, 8).amax(-1)  # noqa: E731
    return most(xv) @ most(wv).T * (7 * 2.0 ** -13)


def e4m3_loss(xv, wv):
    """The same product by product, for few rows: in each eight consecutive
    columns every product but the largest loses less than 2^-13 of the largest
    one's power of two, and no more than itself (cut towards zero)."""
    p = (xv.reshape(xv.shape[0], 1, -1, 8) * wv.reshape(1, wv.shape[0], -1, 8)).abs()
    most = p.amax(-1, keepdim=True)
    grid = torch.exp2(torch.floor(torch.log2(most.clamp(min=2.0 ** -1000)))) * 2.0 ** -13
    return (torch.minimum(p, grid).sum(-1) - torch.minimum(most, grid)[..., 0]).sum(-1)


def gemm(x_q, x_s, w_q, w_s, groups, e4m3=True):
    """[(rows, y, bound)] a group."""
    for e, a, n in groups:
        if n:
            xv, wv = values(x_q[a:a + n], x_s[a:a + n]), values(w_q[e], w_s[e], 128)
            y, d = product(xv, wv, x_q.shape[1])
            yield slice(a, a + n), y, d + _e4m3_products(xv, wv) if e4m3 else d


def swiglu(x_q, x_s, w_q, w_s, groups):
    for sl, y, d in gemm(x_q, x_s, w_q, w_s, groups, e4m3=False):
        i = y.shape[1] // 2
        yield (sl, *silu_mul(y[:, :i], d[:, :i], y[:, i:], d[:, i:]))


def norm(x, residual, gamma, eps):
    """r, n and n's relative bound: a lane adds up to 32 squares, then lanes
    and waves are joined (64 additions deep at most); halved by the root."""
    r = x.double() + (residual.double() if residual is not None else 0.0)
    rf = r.float().double()
    n = rf / torch.sqrt((rf * rf).mean(-1, keepdim=True) + eps) * gamma.double()
    return r, n, 64 * U / 2 + 10 * U


def layer(x, idx, w, w13_q, w13_s, w2_q, w2_s):
    """out and its bound; x [T, H], idx and w [T, k]."""
    T, H = x.shape
    E, _, I = w2_q.shape  # noqa: E741
    out, bound = torch.zeros((T, H), dtype=torch.float64, device=x.device), None
    bound = torch.zeros_like(out)
    mag = torch.zeros_like(out)
    xd = x.double()
    for e in sorted(set(idx.flatten().tolist())):
        if not 0 <= e < E:
            continue
        hit = idx == e
        t = hit.any(1).nonzero().flatten()
        ww = (w.double() * hit).sum(1)[t, None]
        h, dh = product(xd[t], values(w13_q[e], w13_s[e], 128), H)
        a, da = silu_mul(h[:, :I], dh[:, :I], h[:, I:], dh[:, I:])
        # weights of one expert added in float32, the product with them, and
        # the two bf16 parts (half of a bf16 step of half a bf16 step)
        da = da * ww.abs() + (a * ww).abs() * (idx.shape[1] * U + 2.0 ** -16)
        a = a * ww
        w2 = values(w2_q[e], w2_s[e], 128)
        out[t] += a @ w2.T
        m = (a.abs() + da) @ w2.abs().T
        mag[t] += m
        bound[t] += da @ w2.abs().T + m * sum_bound(I, 256)
    return out, bound + mag * (E + 32) * U
