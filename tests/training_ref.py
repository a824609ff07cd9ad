"""Plain float64 forms of the operators that train an expert layer, with
bounds on how far a float32 computation of the same formula may be from them
(units and helpers of expert_ref.py: U = 2^-24 is half a float32 step).

A float32 sum is off by at most U (2U where an addition may truncate) times
the additions a term passes through, times sum |terms|.  A matrix product
adds 32 products in an instruction and joins instructions one after the
other: a term passes through at most 34 additions inside and K / 32 joins.
"""
from __future__ import annotations

import torch

from expert_ref import BF16_HALF, U, check_bf16 as _check_bf16, silu_mul, values


def sum_bound(K):
    return (34 + K / 32 + 8) * 2 * U


def product(x, w, w_t=False):
    """y = x w^T (w [F][K]) or x w (w [K][F]) and its bound."""
    x, w = x.double(), w.double() if w_t else w.double().T
    return x @ w, (x.abs() @ w.abs()) * sum_bound(x.shape[1])


def up(x, w13):
    """(a, bound, [g u], bound) of one expert's rows."""
    h, d = product(x, w13)
    i = h.shape[1] // 2
    a, da = silu_mul(h[:, :i], d[:, :i], h[:, i:], d[:, i:])
    return a, da, h, d


def up_grad(dy, w2, h_q, h_s):
    """(dh, bound, a, bound) of one expert's rows."""
    h = values(h_q, h_s)
    i = h.shape[1] // 2
    g, u = h[:, :i], h[:, i:]
    da, dda = product(dy, w2, True)
    s = torch.sigmoid(g)
    # the exponential's argument is rounded (|g| 2^-23 of it, where it is not
    # negligible against 1), a dozen roundings follow; 1 + g (1 - s) may cancel
    e = (2 * g.abs().clamp(max=110.0) + 16) * U
    D = s * (1 + g * (1 - s))
    eD = e * s * ((1 + g * (1 - s)).abs() + g.abs()) + 0.5 * g.abs() * U
    dg, du, a = da * u * D, da * g * s, g * s * u
    bg = (u * D).abs() * dda + (da * u).abs() * eD + dg.abs() * 4 * U
    bu = (g * s).abs() * dda + du.abs() * e
    return torch.cat((dg, du), 1), torch.cat((bg, bu), 1), a, a.abs() * e


def wgrad(d, x):
    d, x = d.double(), x.double()
    return d.T @ x, (d.abs().T @ x.abs()) * sum_bound(d.shape[0])


def _mean(v):
    return v.mean(-1, keepdim=True)


# Per row: at most 32 additions in a thread, 6 between lanes, 16 between
# waves; roots halve; a value passes through three such sums and some dozens of
# single roundings before it is written.
ROW = 256 * U


def block_norm(x, residual, gp, gate, alpha, gn, eps):
    """r, bound, y, bound (y None without gn)."""
    x, res, gp = x.double(), residual.double(), gp.double()
    gate = 1.0 if gate is None else gate.double()[..., None]
    n1 = x / torch.sqrt(_mean(x * x) + eps) * gp
    r = alpha * res + gate * n1
    br = ROW * ((alpha * res).abs() + (gate * n1).abs())
    if gn is None:
        return r, br, None, None
    i2 = 1 / torch.sqrt(_mean(r * r) + eps)
    y = r * i2 * gn.double()
    return r, br, y, (i2 * gn.double()).abs() * (br + r.abs() * i2 * torch.sqrt(_mean(br * br))) + y.abs() * ROW


def block_norm_grad(dy, dr, x, residual, gp, gate, alpha, gn, eps):
    """{name: (value, bound)}; dy and gn, or dr, may be None."""
    x, res, gp = x.double(), residual.double(), gp.double()
    g = torch.ones(x.shape[:-1], device=x.device, dtype=torch.float64) if gate is None else gate.double()
    g = g[..., None]
    i1 = 1 / torch.sqrt(_mean(x * x) + eps)
    xh = x * i1
    r = alpha * res + g * xh * gp
    ar = (alpha * res).abs() + (g * xh * gp).abs()      # what r's rounding goes by
    i2 = 1 / torch.sqrt(_mean(r * r) + eps)
    d = torch.zeros_like(x) if dr is None else dr.double()
    bd, rh = d.abs(), r * i2
    if dy is not None:
        t = dy.double() * gn.double()
        d = d + i2 * (t - rh * _mean(t * rh))
        grow = 1 + i2 * torch.sqrt(_mean(ar * ar))      # relative change of the root by r's rounding
        bd = bd + i2 * grow * (t.abs() + ar * i2 * _mean(t.abs() * ar * i2) * grow)
    bd = bd * ROW
    dgate = (d * gp * xh).sum(-1)
    bgate = ((bd + ROW * d.abs()) * (gp * xh).abs()).sum(-1)
    dx = i1 * (g * d * gp - xh * g * dgate[..., None] / x.shape[-1])
    bx = i1 * g.abs() * ((bd + ROW * d.abs()) * gp.abs()
                         + xh.abs() * (bgate + ROW * dgate.abs())[..., None] / x.shape[-1])
    out = {"dx": (dx, bx), "dresidual": (alpha * d, abs(alpha) * (bd + ROW * d.abs())), "dgate": (dgate, bgate)}
    rows = x.numel() // x.shape[-1]
    joins = min(rows, 4096) * U                         # a row's share, the workgroups' parts
    flat = lambda v: v.reshape(-1, x.shape[-1]).sum(0)  # noqa: E731
    v, b = g * d * xh, g.abs() * xh.abs() * (bd + ROW * d.abs())
    out["dgamma_post"] = (flat(v), flat(b) + flat(v.abs()) * joins)
    if dy is not None:
        v = dy.double() * rh
        b = dy.double().abs() * ar * i2 * ROW * grow
        out["dgamma_next"] = (flat(v), flat(b) + flat(v.abs()) * joins)
    return out


def check_bf16(got, ref, bound, what=""):
    """As in expert_ref.py, where a result of zeros has no norm to compare with."""
    if bool((ref != 0).any()):
        _check_bf16(got, ref, bound, what)
    else:
        assert bool((got == 0).all()), what


def check_f32(got, ref, bound, what=""):
    lim = bound + U * ref.abs() + 2.0 ** -149
    d = (got.double() - ref).abs()
    bad = ~(d <= lim)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {(d / lim).max().item()}"


def near(got, ref, steps, what=""):
    """`got` within `steps` independent bf16 roundings of the norm: half a step
    spread evenly is 2^-8 / sqrt(3) of the norm at the most."""
    rel = ((got.double() - ref).norm() / ref.norm()).item()
    assert rel <= BF16_HALF / 3 ** 0.5 * steps ** 0.5 * 1.05, f"{what}: {rel} of the norm"
