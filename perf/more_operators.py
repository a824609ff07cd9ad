"""Measured cases of the operators that train an expert layer: the gated
feed-forward block of the experts with an 8-bit checkpoint of its gate and up
rows, its backward pass, the backward pass of the combine, and the norms
after and before a block with the block's gate and residual scale, forwards
and backwards.

`own` False: every operator in elementary torch operations, in 32 bits,
rounded once at the end.  `own` True: the library's calls.
"""
import math

import torch

own = False

BLOCK = 128          # elements that share a scale
E4M3_MAX = 448.0
F8 = torch.float8_e4m3fn
BF = torch.bfloat16
EPS = 1e-6


def listed():
    return [
        # A small model's experts with a handful of rows each (tiny, 5 tokens a rank): the weights' stream.
        {"name": "ffn_tiny", "op": "ffn", "N": 16, "T": 5, "E": 128, "k": 8, "H": 2048, "I": 2048, "skew": False},
        # A Zipf-like load on a quarter of kimi_skewed's experts: some get thousands of rows, others a few.
        {"name": "ffn_skewed", "op": "ffn", "N": 16, "T": 128, "E": 96, "k": 8, "H": 7168, "I": 2048, "skew": True},
        # A training batch: about 2048 rows for each expert.
        {"name": "ffn_heavy", "op": "ffn", "N": 8, "T": 1024, "E": 32, "k": 8, "H": 7168, "I": 2048, "skew": False},
        # Gradients of the small model: the weights and their gradients are all there is to move.
        {"name": "ffn_grad_tiny", "op": "ffn_grad", "N": 16, "T": 5, "E": 128, "k": 8, "H": 2048, "I": 2048,
         "skew": False},
        # One expert that every token visits (a shared expert), an odd number of rows.
        {"name": "ffn_grad_shared", "op": "ffn_grad", "N": 1, "T": 1337, "E": 1, "k": 1, "H": 7168, "I": 2048,
         "skew": False},
        # Gradients of the training batch.
        {"name": "ffn_grad_heavy", "op": "ffn_grad", "N": 8, "T": 1024, "E": 32, "k": 8, "H": 7168, "I": 2048,
         "skew": False},
        # Gradients of the combine at a decode-sized batch (dsv3_decode) and at a training batch (combine_heavy).
        {"name": "combine_grad_small", "op": "combine_grad", "N": 32, "T": 128, "H": 7168, "E": 256, "k": 8},
        {"name": "combine_grad_heavy", "op": "combine_grad", "N": 16, "T": 4096, "H": 7168, "E": 256, "k": 8},
        # The norms around a block: one token (latency), a large batch; their gradients for a small model's odd
        # batch and for the large one.
        {"name": "norm_1", "op": "norm", "N": 1, "T": 1, "H": 7168},
        {"name": "norm_heavy", "op": "norm", "N": 16, "T": 4096, "H": 7168},
        {"name": "norm_grad_odd", "op": "norm_grad", "N": 3, "T": 333, "H": 2048},
        {"name": "norm_grad_heavy", "op": "norm_grad", "N": 16, "T": 4096, "H": 7168},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_grad", "ffn_grad", "combine_grad", "norm", "norm_grad"])
    n = rng.choice([1, 2, 4, 8, 16])
    if op in ("norm", "norm_grad"):
        return {"op": op, "N": n, "T": _spread(rng, 1, 65536 // n), "H": 128 * rng.randint(1, 56)}
    e = n * rng.randint(1, 64 // n)
    k = rng.randint(1, min(8, e))
    if op == "combine_grad":
        return {"op": op, "N": n, "T": _spread(rng, 1, 65536 // n), "H": 128 * rng.randint(1, 56), "E": e, "k": k}
    e = min(e, 32 // n * n)
    k = min(k, e)
    return {"op": op, "N": n, "T": _spread(rng, 1, 65536 // n // k), "E": e, "k": k, "H": 128 * rng.randint(1, 56),
            "I": 128 * rng.randint(1, 16), "skew": rng.random() < 0.4}


# --------------------------------------------------------------- inputs

def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _bf16(shape, gen, std=1.0):
    """Normal bf16 values, made in parts of about 2^27."""
    x = torch.empty(shape, dtype=BF, device="cuda")
    flat = x.view(shape[0], -1)
    step = max(1, (1 << 27) // max(1, flat.shape[1]))
    for a in range(0, shape[0], step):
        b = min(shape[0], a + step)
        flat[a:b] = _normal((b - a, flat.shape[1]), gen, std)
    return x


def _topk(tokens, experts, k, skew, gen):
    logits = _normal((tokens, experts), gen)
    if skew:
        logits -= torch.log(torch.randperm(experts, generator=gen, device="cuda") + 1.0)
    v, i = logits.topk(k, 1)
    return i.to(torch.int32), torch.softmax(v, 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    empty = lambda *shape, t=BF: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    if own:
        import combine_lds_atomic_amd as moe
        s["shape"] = moe.shape(c["N"], c["T"], c["H"], c.get("E", c["N"]), c.get("k", 1))
    N, T, H = c["N"], c["T"], c["H"]
    if c["op"] in ("norm", "norm_grad"):
        s["x"], s["residual"] = _bf16((N, T, H), gen, 0.5), _bf16((N, T, H), gen, 3.0)
        s["gamma_post"], s["gamma_next"] = ((1 + _normal((H,), gen, 0.1)).to(BF) for _ in range(2))
        s["gate"] = torch.sigmoid(_normal((N, T), gen))     # as a router's output layer gives it
        s["alpha"] = 0.8125
        if c["op"] == "norm_grad":
            s["dy"], s["dres"] = _bf16((N, T, H), gen), _bf16((N, T, H), gen)
        if own and c["op"] == "norm":
            s["out"] = [empty(N, T, H), empty(N, T, H)]
        elif own:
            s["out"] = [empty(N, T, H), empty(N, T, H), empty(N, T, t=torch.float32), empty(H, t=torch.float32),
                        empty(H, t=torch.float32)]
            s["ws"] = empty(moe.moe_block_norm_grad_workspace_bytes(s["shape"]), t=torch.uint8)
        return s
    E, k = c["E"], c["k"]
    rows = N * T * k
    idx, w = _topk(N * T, E, k, c.get("skew", False), gen)
    if c["op"] == "combine_grad":
        s["idx"], s["w"] = idx.view(N, T, k), w.view(N, T, k).contiguous()
        # slots in the order of their expert-major rows
        s["order"] = torch.sort(idx.reshape(-1), stable=True).indices
        s["dout"], s["y_em"] = _bf16((N, T, H), gen), _bf16((rows, H), gen)
        if own:
            L = E // N
            s["ws"] = empty(moe.moe_workspace_bytes(s["shape"]), t=torch.uint8)
            s["send_pos"], s["row_src"] = empty(N, T, k, t=torch.int32), empty(rows, t=torch.int32)
            s["out"] = [empty(rows, H), empty(N, T, k, t=torch.float32)]
            moe.moe_workspace_init(s["shape"], s["ws"])
            moe.moe_dispatch_direct(s["shape"], None, s["idx"], None, None, s["send_pos"],
                                    empty(N, L + 1, t=torch.int32), s["row_src"], s["ws"])
        return s
    I = c["I"]  # noqa: E741
    counts = torch.bincount(idx.reshape(-1).long(), minlength=E)
    off = torch.zeros((N, E // N + 1), dtype=torch.int64, device="cuda")
    off[:, 1:] = counts.view(N, E // N).cumsum(1)
    s["exp_off"], s["counts"] = off.to(torch.int32), counts.tolist()
    s["x"] = _bf16((rows, H), gen)
    s["w13"], s["w2"] = _bf16((E, 2 * I, H), gen, H ** -0.5), _bf16((E, H, I), gen, I ** -0.5)
    if c["op"] == "ffn_grad":
        s["dy"] = _bf16((rows, H), gen)
        h = _bf16((rows, 2 * I), gen).float().view(rows, -1, BLOCK)
        s["h_s"] = h.abs().amax(-1) / E4M3_MAX
        s["h_q"] = (h / s["h_s"].unsqueeze(-1)).to(F8).view(rows, 2 * I).view(torch.uint8)
        if own:
            s["out"] = {"dh": empty(rows, 2 * I), "a": empty(rows, I), "dx": empty(rows, H),
                        "dw13": empty(E, 2 * I, H), "dw2": empty(E, H, I)}
    elif own:
        s["out"] = {"a": empty(rows, I), "h_q": empty(rows, 2 * I, t=torch.uint8),
                    "h_s": empty(rows, 2 * I // BLOCK, t=torch.float32), "y": empty(rows, H)}
    return s


# --------------------------------------------------------------- plain forms

def _quantise(v):
    """e4m3 bytes and scales (amax / 448) of fp32 rows; a block of zeros has scale 0."""
    b = v.view(*v.shape[:-1], -1, BLOCK)
    s = b.abs().amax(-1) / E4M3_MAX
    q = (b / torch.where(s == 0, 1.0, s).unsqueeze(-1)).to(F8)
    return q.view(v.shape), s


def _ffn(s):
    """Each expert's block over its own rows.  The groups are ragged, so this is one pass a group."""
    c = s["case"]
    I, rows = c["I"], s["x"].shape[0]  # noqa: E741
    y = torch.empty_like(s["x"])
    q = torch.empty((rows, 2 * I), dtype=F8, device="cuda")
    sc = torch.empty((rows, 2 * I // BLOCK), device="cuda")
    a = 0
    for e, n in enumerate(s["counts"]):
        if n:
            h = s["x"][a:a + n].float() @ s["w13"][e].float().t()
            q[a:a + n], sc[a:a + n] = _quantise(h)
            act = h[:, :I] / (1 + torch.exp(-h[:, :I])) * h[:, I:]
            y[a:a + n] = act @ s["w2"][e].float().t()
        a += n
    return {"y": y, "h_q": q, "h_s": sc}


def _ffn_grad(s):
    I = s["case"]["I"]  # noqa: E741
    dx, dw13, dw2 = torch.empty_like(s["x"]), torch.zeros_like(s["w13"]), torch.zeros_like(s["w2"])
    a = 0
    for e, n in enumerate(s["counts"]):
        if n:
            x, dy = s["x"][a:a + n].float(), s["dy"][a:a + n].float()
            h = s["h_q"][a:a + n].view(F8).float().view(n, -1, BLOCK) * s["h_s"][a:a + n].unsqueeze(-1)
            h = h.view(n, 2 * I)
            g, u = h[:, :I], h[:, I:]
            da, sig = dy @ s["w2"][e].float(), 1 / (1 + torch.exp(-g))
            dh = torch.cat((da * u * sig * (1 + g * (1 - sig)), da * g * sig), 1)
            dx[a:a + n] = dh @ s["w13"][e].float()
            dw13[e] = dh.t() @ x
            dw2[e] = dy.t() @ (g * sig * u)
        a += n
    return {"dx": dx, "dw13": dw13, "dw2": dw2}


def _combine_grad(s):
    H, k = s["case"]["H"], s["case"]["k"]
    order = s["order"]
    d = s["dout"].view(-1, H)[order // k].float()
    dw = torch.empty_like(s["w"]).view(-1)
    dw[order] = (d * s["y_em"].float()).sum(-1)
    return {"dy_em": d.mul_(s["w"].view(-1)[order].unsqueeze(-1)).to(BF), "dw": dw.view(s["w"].shape)}


def _unit(v):
    """v over its root mean square, and the reciprocal of that."""
    inv = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    return v * inv, inv


def _norm(s):
    xh, _ = _unit(s["x"].float())
    r = s["alpha"] * s["residual"].float() + s["gate"].unsqueeze(-1) * (xh * s["gamma_post"].float())
    return {"res": r.to(BF), "y": (_unit(r)[0] * s["gamma_next"].float()).to(BF)}


def _norm_grad(s):
    gp, gn, gate, dy = s["gamma_post"].float(), s["gamma_next"].float(), s["gate"].unsqueeze(-1), s["dy"].float()
    xh, i1 = _unit(s["x"].float())
    rh, i2 = _unit(s["alpha"] * s["residual"].float() + gate * (xh * gp))
    t = dy * gn
    dr = s["dres"].float() + i2 * (t - rh * (t * rh).mean(-1, keepdim=True))
    t = gate * dr
    dx = i1 * (t * gp - xh * (t * gp * xh).mean(-1, keepdim=True))
    return {"dx": dx.to(BF), "dresidual": (s["alpha"] * dr).to(BF), "dgate": (dr * xh * gp).sum(-1),
            "dgamma_post": (t * xh).sum((0, 1)), "dgamma_next": (dy * rh).sum((0, 1))}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"ffn": _ffn, "ffn_grad": _ffn_grad, "combine_grad": _combine_grad, "norm": _norm,
                "norm_grad": _norm_grad}[op](s)
    import combine_lds_atomic_amd as moe
    sh, out, H, I = s["shape"], s["out"], c["H"], c.get("I")  # noqa: E741
    if op == "ffn":
        moe.moe_ffn_up(sh, s["x"], s["w13"], s["exp_off"], H, I, out["a"], out["h_q"], out["h_s"])
        moe.moe_grouped_gemm_bf16(sh, out["a"], s["w2"], s["exp_off"], I, H, False, out["y"])
        return {"y": out["y"], "h_q": out["h_q"].view(F8), "h_s": out["h_s"]}
    if op == "ffn_grad":
        moe.moe_ffn_up_grad(sh, s["dy"], s["w2"], s["h_q"], s["h_s"], s["exp_off"], H, I, out["dh"], out["a"])
        moe.moe_grouped_gemm_bf16(sh, out["dh"], s["w13"], s["exp_off"], 2 * I, H, True, out["dx"])
        moe.moe_grouped_wgrad(sh, out["dh"], s["x"], s["exp_off"], 2 * I, H, out["dw13"])
        moe.moe_grouped_wgrad(sh, s["dy"], out["a"], s["exp_off"], H, I, out["dw2"])
        return {"dx": out["dx"], "dw13": out["dw13"], "dw2": out["dw2"]}
    if op == "combine_grad":
        moe.moe_combine_grad(sh, s["dout"], s["y_em"], s["idx"], s["send_pos"], s["w"], s["row_src"], s["ws"], *out)
        return {"dy_em": out[0], "dw": out[1]}
    if op == "norm":
        moe.moe_block_norm(sh, s["x"], s["residual"], s["gamma_post"], s["gate"], s["alpha"], s["gamma_next"], EPS,
                           *out)
        return dict(zip(("res", "y"), out))
    moe.moe_block_norm_grad(sh, s["dy"], s["dres"], s["x"], s["residual"], s["gamma_post"], s["gate"], s["alpha"],
                            s["gamma_next"], EPS, *out, s["ws"])
    return dict(zip(("dx", "dresidual", "dgate", "dgamma_post", "dgamma_next"), out))


# --------------------------------------------------------------- work and the 64-bit results

def _active(c):
    """Experts that N * T tokens with k distinct experts each reach on average, for an even load."""
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** (c["N"] * c["T"]))


def work(case):
    c = case
    n, H = c["N"] * c["T"], c["H"]
    if c["op"] == "norm":
        return {"bytes": n * (8 * H + 4) + 4 * H, "flops": 12 * n * H}
    if c["op"] == "norm_grad":
        return {"bytes": n * (12 * H + 8) + 12 * H, "flops": 40 * n * H}
    rows = n * c["k"]
    if c["op"] == "combine_grad":
        return {"bytes": n * 2 * H + rows * (4 * H + 16), "flops": 3 * rows * H}
    I, active = c["I"], _active(c)  # noqa: E741
    weights = 3 * H * I * 2
    h = rows * 2 * I * (1 + 4 / BLOCK)
    if c["op"] == "ffn":
        return {"bytes": active * weights + rows * 4 * H + h, "flops": 6 * rows * H * I}
    return {"bytes": active * weights + c["E"] * weights + rows * 6 * H + h, "flops": 12 * rows * H * I}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    D = torch.float64
    if c["op"] in ("norm", "norm_grad"):
        parts = []
        gp, gn = s["gamma_post"].to(D), s["gamma_next"].to(D)
        for i in range(c["N"]):        # rank by rank: the 64-bit rows are large
            x, res, g = s["x"][i].to(D), s["residual"][i].to(D), s["gate"][i].to(D)[:, None]
            n1 = (x.pow(2).sum(1, keepdim=True) / c["H"] + EPS).sqrt()
            r = res * s["alpha"] + x / n1 * gp * g
            n2 = (r.pow(2).sum(1, keepdim=True) / c["H"] + EPS).sqrt()
            if c["op"] == "norm":
                parts.append((r, r / n2 * gn))
                continue
            dy = s["dy"][i].to(D)
            # d(r / n2): the part along r is taken out
            along = (dy * gn * r).sum(1, keepdim=True) / (c["H"] * n2 ** 3)
            dr = s["dres"][i].to(D) + dy * gn / n2 - r * along
            dg = (dr * gp * x / n1).sum(1)
            dx = g * (dr * gp / n1 - x * (dr * gp * x).sum(1, keepdim=True) / (c["H"] * n1 ** 3))
            parts.append((dx, dr * s["alpha"], dg, (dr * g * x / n1).sum(0), (dy * r / n2).sum(0)))
        v = [torch.stack(p) for p in zip(*parts)]
        if c["op"] == "norm":
            return {"res": v[0], "y": v[1]}
        return {"dx": v[0], "dresidual": v[1], "dgate": v[2], "dgamma_post": v[3].sum(0), "dgamma_next": v[4].sum(0)}
    if c["op"] == "combine_grad":
        rows, k, H = s["y_em"].shape[0], c["k"], c["H"]
        dy = torch.empty((rows, H), dtype=D, device="cuda")
        dw = torch.empty(rows, dtype=D, device="cuda")
        for a in range(0, rows, 1 << 16):
            slot = s["order"][a:a + (1 << 16)]
            d = s["dout"].reshape(-1, H)[torch.div(slot, k, rounding_mode="floor")].to(D)
            dy[a:a + (1 << 16)] = d * s["w"].reshape(-1)[slot].to(D)[:, None]
            dw[slot] = torch.einsum("ij,ij->i", d, s["y_em"][a:a + (1 << 16)].to(D))
        return {"dy_em": dy, "dw": dw.view(s["w"].shape)}

    I, H = c["I"], c["H"]  # noqa: E741
    rows = s["x"].shape[0]
    new = lambda *shape: torch.zeros(shape, dtype=D, device="cuda")  # noqa: E731
    ends = torch.tensor(s["counts"]).cumsum(0).tolist()
    if c["op"] == "ffn":
        y, q, sc = new(rows, H), new(rows, 2 * I), new(rows, 2 * I // BLOCK)
        for e, b in enumerate(ends):
            r = slice(b - s["counts"][e], b)
            x, w = s["x"][r].to(D), s["w13"][e].to(D)
            g, u = x @ w[:I].T, x @ w[I:].T
            y[r] = (torch.sigmoid(g) * g * u) @ s["w2"][e].to(D).T
            h = torch.cat((g, u), 1).reshape(-1, BLOCK)
            m = h.abs().max(1).values / E4M3_MAX
            sc[r] = m.view(-1, 2 * I // BLOCK)
            q[r] = (h / m.clamp(min=1e-300)[:, None]).float().to(F8).to(D).view(-1, 2 * I)
        return {"y": y, "h_q": q, "h_s": sc}
    dx, dw13, dw2 = new(rows, H), new(c["E"], 2 * I, H), new(c["E"], H, I)
    for e, b in enumerate(ends):
        r = slice(b - s["counts"][e], b)
        x, dy, w13, w2 = (v.to(D) for v in (s["x"][r], s["dy"][r], s["w13"][e], s["w2"][e]))
        h = s["h_q"][r].view(F8).to(D) * s["h_s"][r].to(D).repeat_interleave(BLOCK, 1)
        g, u = h[:, :I], h[:, I:]
        t, da = torch.sigmoid(g), dy @ w2
        dg, du = da * u * (t + g * t * torch.sigmoid(-g)), da * g * t
        dx[r] = dg @ w13[:I] + du @ w13[I:]
        dw13[e, :I], dw13[e, I:], dw2[e] = dg.T @ x, du.T @ x, dy.T @ (g * t * u)
    return {"dx": dx, "dw13": dw13, "dw2": dw2}
