"""Measured cases of the expert layer's operators: the RMS norm with the
residual's addition and an 8-bit output, the block-scaled fp8 products over
the expert-major rows that dispatch writes (plain, and with the SwiGLU and
requantising epilogue), and the whole layer for a few tokens.

`own` False: every operator in elementary torch operations, in 32 bits,
rounded once at the end.  `own` True: the library's calls.
"""
import math

import torch

own = False

BLOCK = 128          # elements that share a scale
E4M3_MAX = 448.0
F8 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # One decode step of a single token: the call is latency.
        {"name": "norm_1", "op": "norm", "N": 1, "T": 1, "H": 7168},
        # A decode batch over 32 ranks, 128 tokens each (dsv3_decode).
        {"name": "norm_decode", "op": "norm", "N": 32, "T": 128, "H": 7168},
        # A large batch over 16 ranks, 4096 tokens each (combine_heavy).
        {"name": "norm_heavy", "op": "norm", "N": 16, "T": 4096, "H": 7168},
        # The gate/up product of a decode batch: about 128 rows for each of 256 experts.
        {"name": "swiglu_decode", "op": "swiglu", "N": 32, "T": 128, "E": 256, "k": 8, "K": 7168, "F": 2048, "skew": False},
        # The same under a Zipf-like load (kimi_skewed): some experts get thousands of rows, others a few.
        {"name": "swiglu_skewed", "op": "swiglu", "N": 64, "T": 128, "E": 384, "k": 8, "K": 7168, "F": 2048, "skew": True},
        # The gate/up product of a large batch: about 2048 rows for each expert.
        {"name": "swiglu_heavy", "op": "swiglu", "N": 16, "T": 4096, "E": 256, "k": 8, "K": 7168, "F": 2048, "skew": False},
        # A small model's experts with a handful of rows each (tiny, 5 tokens a rank).
        {"name": "gemm_tiny", "op": "gemm", "N": 16, "T": 5, "E": 128, "k": 8, "K": 2048, "F": 2048, "skew": False},
        # One expert that every token visits (a shared expert), an odd number of rows.
        {"name": "gemm_shared", "op": "gemm", "N": 1, "T": 1337, "E": 1, "k": 1, "K": 7168, "F": 4096, "skew": False},
        # The down product of a large batch.
        {"name": "gemm_heavy", "op": "gemm", "N": 16, "T": 4096, "E": 256, "k": 8, "K": 2048, "F": 7168, "skew": False},
        # The whole layer: one token, a small batch, and the largest batch the call takes.
        {"name": "layer_1", "op": "layer", "N": 1, "T": 1, "E": 256, "k": 8, "H": 7168, "I": 2048},
        {"name": "layer_13", "op": "layer", "N": 1, "T": 13, "E": 256, "k": 8, "H": 7168, "I": 2048},
        {"name": "layer_64", "op": "layer", "N": 8, "T": 8, "E": 128, "k": 8, "H": 2048, "I": 2048},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "swiglu", "gemm", "layer"])
    if op == "norm":
        n = rng.choice([1, 2, 4, 8, 16])
        return {"op": op, "N": n, "T": _spread(rng, 1, 4096), "H": 128 * rng.randint(1, 64)}
    if op == "layer":
        n, e = rng.choice([1, 2, 4, 8]), 8 * rng.randint(1, 32)
        return {"op": op, "N": n, "T": _spread(rng, 1, 64 // n), "E": e, "k": rng.randint(1, 8),
                "H": 128 * rng.randint(4, 56), "I": 128 * rng.randint(2, 16)}
    n, f = rng.choice([1, 2, 4, 8]), rng.randint(2, 16)
    return {"op": op, "N": n, "T": _spread(rng, 1, 4096), "E": n * rng.randint(1, 128 // n), "k": 1 if n == 1 else 2,
            "K": 128 * rng.randint(2, 56), "F": 128 * f if op == "swiglu" else 16 * rng.randint(8, 448),
            "skew": rng.random() < 0.4}


# --------------------------------------------------------------- inputs

def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _rows_q(rows, cols, gen):
    """Token rows as dispatch stores them: e4m3 bytes and one scale for each 128 elements."""
    q = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, cols // BLOCK), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // cols)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        x = _normal((b - a, cols // BLOCK, BLOCK), gen)
        s[a:b] = x.abs().amax(-1) / E4M3_MAX
        q[a:b] = (x / s[a:b, :, None]).to(F8).view(torch.uint8).reshape(b - a, cols)
    return q, s


def _weights_q(experts, out, cols, gen):
    """Expert weights in e4m3 with one scale for each 128 x 128 block (the last row block may be short)."""
    nb, kb = -(-out // BLOCK), cols // BLOCK
    q = torch.empty((experts, out, cols), dtype=torch.uint8, device="cuda")
    s = torch.empty((experts, nb, kb), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (nb * BLOCK * cols))
    for a in range(0, experts, step):
        b = min(experts, a + step)
        w = _normal((b - a, nb, BLOCK, kb, BLOCK), gen, cols ** -0.5)
        s[a:b] = w.abs().amax((2, 4)) / E4M3_MAX
        w = (w / s[a:b, :, None, :, None]).to(F8).view(torch.uint8)
        q[a:b] = w.reshape(b - a, nb * BLOCK, cols)[:, :out]
    return q, s


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
    if c["op"] == "norm":
        shape = (c["N"], c["T"], c["H"])
        s["x"], s["residual"] = (_normal(shape, gen, d).to(torch.bfloat16) for d in (1.0, 4.0))
        s["gamma"] = (1 + _normal((c["H"],), gen, 0.1)).to(torch.bfloat16)
        if own:
            import combine_lds_atomic_amd as moe
            s["shape"] = moe.shape(c["N"], c["T"], c["H"], c["N"], 1)
            s["out"] = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            s["out"] += [torch.empty(shape, dtype=torch.uint8, device="cuda"),
                         torch.empty((c["N"], c["T"], c["H"] // BLOCK), dtype=torch.float32, device="cuda")]
        return s
    if c["op"] == "layer":
        H, I, tokens = c["H"], c["I"], c["N"] * c["T"]
        s["x"] = _normal((c["N"], c["T"], H), gen).to(torch.bfloat16)
        idx, w = _topk(tokens, c["E"], c["k"], False, gen)
        s["idx"], s["w"] = idx.view(c["N"], c["T"], -1), w.view(c["N"], c["T"], -1)
        s["w13_q"], s["w13_s"] = _weights_q(c["E"], 2 * I, H, gen)
        s["w2_q"], s["w2_s"] = _weights_q(c["E"], H, I, gen)
        if own:
            import combine_lds_atomic_amd as moe
            s["shape"] = moe.shape(c["N"], c["T"], H, c["E"], c["k"])
            s["ws"] = torch.empty(moe.moe_layer_ll_workspace_bytes(s["shape"], I), dtype=torch.uint8, device="cuda")
            s["out"] = torch.empty((c["N"], c["T"], H), dtype=torch.bfloat16, device="cuda")
            s["flags"] = torch.empty(1, dtype=torch.int32, device="cuda")
        return s
    rows, N, E = c["N"] * c["T"] * c["k"], c["N"], c["E"]
    idx, _ = _topk(N * c["T"], E, c["k"], c["skew"], gen)
    counts = torch.bincount(idx.reshape(-1).long(), minlength=E)
    off = torch.zeros((N, E // N + 1), dtype=torch.int64, device="cuda")
    off[:, 1:] = counts.view(N, E // N).cumsum(1)
    s["exp_off"], s["counts"] = off.to(torch.int32), counts.tolist()
    s["x_q"], s["x_s"] = _rows_q(rows, c["K"], gen)
    out = 2 * c["F"] if c["op"] == "swiglu" else c["F"]
    s["w_q"], s["w_s"] = _weights_q(E, out, c["K"], gen)
    if own:
        import combine_lds_atomic_amd as moe
        s["shape"] = moe.shape(N, c["T"], c["K"], E, c["k"])
        if c["op"] == "swiglu":
            s["out"] = (torch.empty((rows, c["F"]), dtype=torch.uint8, device="cuda"),
                        torch.empty((rows, c["F"] // BLOCK), dtype=torch.float32, device="cuda"))
        else:
            s["out"] = torch.empty((rows, c["F"]), dtype=torch.bfloat16, device="cuda")
    return s


# --------------------------------------------------------------- plain forms

def _values(q, s, rows_per_scale=1):
    """fp32 values of e4m3 bytes [..., R, C] with scales [..., R / rows_per_scale, C / 128]."""
    v = q.view(F8).float()
    if rows_per_scale > 1:
        s = s.repeat_interleave(rows_per_scale, -2)[..., :q.shape[-2], :]
    return v.view(*q.shape[:-1], -1, BLOCK).mul_(s.unsqueeze(-1)).view(q.shape)


def _quantise(v):
    """e4m3 bytes and scales (amax / 448) of fp32 rows; a block of zeros has scale 0."""
    b = v.view(*v.shape[:-1], -1, BLOCK)
    s = b.abs().amax(-1) / E4M3_MAX
    q = (b / torch.where(s == 0, 1.0, s).unsqueeze(-1)).to(F8)
    return q.view(v.shape), s


def _silu_mul(gate, up):
    return gate / (1 + torch.exp(-gate)) * up


def _norm(s):
    r = s["x"].float() + s["residual"].float()
    n = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    q, sc = _quantise(n)
    return {"res": r.to(torch.bfloat16), "y": n.to(torch.bfloat16), "y_q": q, "y_s": sc}


def _products(s):
    """Each expert's product over its own rows.  The groups are ragged, so this is one product a group."""
    c = s["case"]
    swiglu = c["op"] == "swiglu"
    rows = s["x_q"].shape[0]
    y = torch.empty((rows, c["F"]), dtype=F8 if swiglu else torch.bfloat16, device="cuda")
    sc = torch.empty((rows, c["F"] // BLOCK), device="cuda") if swiglu else None
    a = 0
    for e, n in enumerate(s["counts"]):
        if n:
            w = _values(s["w_q"][e], s["w_s"][e], BLOCK)
            v = _values(s["x_q"][a:a + n], s["x_s"][a:a + n]) @ w.t()
            if swiglu:
                y[a:a + n], sc[a:a + n] = _quantise(_silu_mul(v[:, :c["F"]], v[:, c["F"]:]))
            else:
                y[a:a + n] = v
        a += n
    return {"a_q": y, "a_s": sc} if swiglu else y


def _layer(s):
    c = s["case"]
    I, tokens, k = c["I"], c["N"] * c["T"], c["k"]
    x = s["x"].float().view(tokens, -1)
    idx, w = s["idx"].view(-1).long(), s["w"].view(tokens, k, 1)
    if tokens * k <= c["E"]:        # few slots: each slot's own weights
        pick = lambda n: _values(s[n + "_q"][idx], s[n + "_s"][idx], BLOCK)  # noqa: E731
        h = (pick("w13") @ x.repeat_interleave(k, 0).unsqueeze(-1)).squeeze(-1)
        y = (pick("w2") @ _silu_mul(h[:, :I], h[:, I:]).unsqueeze(-1)).squeeze(-1)
    else:                           # more slots than experts: every expert on every token, then the chosen ones
        h = x @ _values(s["w13_q"], s["w13_s"], BLOCK).transpose(1, 2)
        y = _silu_mul(h[..., :I], h[..., I:]) @ _values(s["w2_q"], s["w2_s"], BLOCK).transpose(1, 2)
        y = y[idx, torch.arange(tokens, device="cuda").repeat_interleave(k)]
    return (y.view(tokens, k, -1) * w).sum(1).to(torch.bfloat16).view(s["x"].shape)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _norm, "swiglu": _products, "gemm": _products, "layer": _layer}[c["op"]](s)
    import combine_lds_atomic_amd as moe
    if c["op"] == "norm":
        res, y, q, sc = s["out"]
        moe.moe_rmsnorm_quant(s["shape"], s["x"], s["residual"], s["gamma"], EPS, res, y, q, sc)
        return {"res": res, "y": y, "y_q": q.view(F8), "y_s": sc}
    if c["op"] == "layer":
        moe.moe_layer_ll(s["shape"], s["x"], s["idx"], s["w"], s["w13_q"], s["w13_s"], s["w2_q"], s["w2_s"], c["I"],
                         s["out"], s["flags"], s["ws"])
        return s["out"]
    if c["op"] == "swiglu":
        q, sc = s["out"]
        moe.moe_grouped_gemm_swiglu(s["shape"], s["x_q"], s["x_s"], s["w_q"], s["w_s"], s["exp_off"], c["K"], c["F"],
                                    q, sc)
        return {"a_q": q.view(F8), "a_s": sc}
    moe.moe_grouped_gemm(s["shape"], s["x_q"], s["x_s"], s["w_q"], s["w_s"], s["exp_off"], c["K"], c["F"], s["out"])
    return s["out"]


# --------------------------------------------------------------- work and the 64-bit results

def _active(c, draws):
    """Experts that `draws` tokens with k distinct experts each reach on average, for an even load."""
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** draws)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["N"] * c["T"]
        return {"bytes": n * (c["H"] * 9 + c["H"] // 32) + 2 * c["H"], "flops": 6 * n * c["H"]}
    if c["op"] == "layer":
        n = c["N"] * c["T"]
        w = 3 * c["H"] * c["I"]
        return {"bytes": _active(c, n) * w * (1 + 4 / BLOCK ** 2) + n * (4 * c["H"] + 8 * c["k"]),
                "flops": 2 * n * c["k"] * w}
    rows = c["N"] * c["T"] * c["k"]
    out = 2 * c["F"] if c["op"] == "swiglu" else c["F"]
    experts = _active(c, c["N"] * c["T"])
    b = rows * c["K"] * (1 + 4 / BLOCK) + experts * out * c["K"] * (1 + 4 / BLOCK ** 2)
    b += rows * (c["F"] * (1 + 4 / BLOCK) if c["op"] == "swiglu" else 2 * c["F"])
    return {"bytes": b, "flops": 2 * rows * c["K"] * out}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]

    def wide(q, sc, r):
        m = q.view(F8).double()
        i = torch.arange(m.shape[0], device="cuda") // r
        j = torch.arange(m.shape[1], device="cuda") // BLOCK
        return m * sc.double()[i][:, j]

    def eight(v):
        b = v.reshape(-1, BLOCK)
        sc = b.abs().max(1).values / E4M3_MAX
        q = torch.where(sc[:, None] > 0, b / sc[:, None], torch.zeros_like(b)).float().to(F8)
        return q.view(v.shape), sc.view(*v.shape[:-1], -1)

    def ffn(x, e, I):
        h = x @ wide(s["w13_q"][e], s["w13_s"][e], BLOCK).T
        return (torch.sigmoid(h[:, :I]) * h[:, :I] * h[:, I:]) @ wide(s["w2_q"][e], s["w2_s"][e], BLOCK).T

    if c["op"] == "norm":
        rows = []
        for x, res in zip(s["x"], s["residual"]):
            r = x.double() + res.double()
            n = r / ((r * r).sum(-1, keepdim=True) / c["H"] + EPS).sqrt() * s["gamma"].double()
            rows.append((r, n, *eight(n)))
        return dict(zip(("res", "y", "y_q", "y_s"), (torch.stack(v) for v in zip(*rows))))
    if c["op"] == "layer":
        x, idx = s["x"].double().flatten(0, 1), s["idx"].flatten(0, 1)
        out = torch.zeros_like(x)
        for e in idx.unique().tolist():
            t, j = (idx == e).nonzero(as_tuple=True)
            out[t] += s["w"].flatten(0, 1)[t, j, None].double() * ffn(x[t], e, c["I"])
        return out.view(s["x"].shape)
    parts, a = [], 0
    for e, n in enumerate(s["counts"]):
        w = wide(s["w_q"][e], s["w_s"][e], BLOCK)
        for b in range(a, a + n, 1 << 15):
            m = min(a + n, b + (1 << 15))
            v = wide(s["x_q"][b:m], s["x_s"][b:m], 1) @ w.T
            if c["op"] == "gemm":
                parts.append((v,))
            else:
                g, u = v.chunk(2, 1)
                parts.append(eight(g * torch.sigmoid(g) * u))
        a += n
    cols = [torch.cat(v) for v in zip(*parts)]
    return cols[0] if c["op"] == "gemm" else {"a_q": cols[0], "a_s": cols[1]}
