"""The expert layer's operators on the GPU against plain float64 forms
(tests/expert_ref.py), at the sizes, layouts and values where they can go
wrong, and a run of them together as a layer."""
import pytest
import torch

import combine_lds_atomic_amd as moe
import expert_ref as X
import workloads as W

pytestmark = pytest.mark.gpu

from gpu_harness import log  # noqa: E402


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("H", [128, 384, 512, 640, 2048, 7168, 8192, 8320, 16384, 20480, 32768])
@pytest.mark.parametrize("rows", [1, 5])
def test_norm_sizes(H, rows):
    log(f"norm H={H} rows={rows}")
    g = gen(H + rows)
    sh = moe.shape(1, rows, H, 1, 1)
    x, res = (torch.randn((1, rows, H), generator=g, device="cuda").mul(s).bfloat16() for s in (1.0, 5.0))
    gamma = torch.randn(H, generator=g, device="cuda").bfloat16()
    res_out, y = torch.empty_like(x), torch.empty_like(x)
    q = torch.empty((1, rows, H), dtype=torch.uint8, device="cuda")
    s = torch.empty((1, rows, H // 128), device="cuda")
    moe.moe_rmsnorm_quant(sh, x, res, gamma, 1e-5, res_out, y, q, s)
    r, n, rel = X.norm(x[0], res[0], gamma, 1e-5)
    X.check_bf16(res_out[0], r, r.abs() * X.U, "r")
    X.check_bf16(y[0], n, n.abs() * rel, "y")
    X.check_quantised(q[0], s[0], n, n.abs() * rel, "q")
    # the choice of outputs changes none of them
    y2, q2, s2 = torch.empty_like(y), torch.empty_like(q), torch.empty_like(s)
    moe.moe_rmsnorm_quant(sh, x, res, gamma, 1e-5, None, y2, None, None)
    moe.moe_rmsnorm_quant(sh, x, res, gamma, 1e-5, None, None, q2, s2)
    assert torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("N,T,H", [(3, 7, 256), (2, 300, 1024), (8, 33, 7168)])
def test_norm_many_rows_no_residual_and_in_place(N, T, H):
    log(f"norm N={N} T={T} H={H}")
    g = gen(T)
    sh = moe.shape(N, T, H, N, 1)
    x = torch.randn((N, T, H), generator=g, device="cuda").bfloat16()
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    moe.moe_rmsnorm_quant(sh, x, None, gamma, 1e-6, None, y, None, None)
    _, n, rel = X.norm(x, None, gamma, 1e-6)
    X.check_bf16(y, n, n.abs() * rel)
    # residual stream updated in place, norm written over its input
    a, b = x.clone(), torch.randn_like(x)
    r, n, rel = X.norm(a, b, gamma, 1e-6)
    moe.moe_rmsnorm_quant(sh, a, b, gamma, 1e-6, b, a, None, None)
    X.check_bf16(b, r, r.abs() * X.U)
    X.check_bf16(a, n, n.abs() * rel)


def test_norm_values():
    """A row of zeros, tiny and large values, an infinity and a NaN; each row
    on its own."""
    H = 512
    sh = moe.shape(1, 6, H, 1, 1)
    x = torch.zeros((1, 6, H), dtype=torch.bfloat16, device="cuda")
    x[0, 1] = 1e-30
    x[0, 2] = 1e15
    x[0, 3] = 1.0
    x[0, 3, 200] = float("inf")
    x[0, 4] = 1.0
    x[0, 4, 3] = float("nan")
    x[0, 5, :128] = 2.0          # further blocks are zeros
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    q, s = torch.empty((1, 6, H), dtype=torch.uint8, device="cuda"), torch.empty((1, 6, 4), device="cuda")
    moe.moe_rmsnorm_quant(sh, x, None, gamma, 1e-6, None, y, q, s)
    y, q, s = y[0].float().cpu(), q[0].cpu(), s[0].cpu()
    assert (y[0] == 0).all() and (q[0] == 0).all() and (s[0] == 0).all()
    assert torch.allclose(y[1], torch.full((H,), 1e-27), rtol=2.0 ** -7)
    assert (y[2] == 1).all()
    assert y[3, 200].isnan() and (y[3, :200] == 0).all()       # 1 / infinity
    assert s[3, 1].isnan() and (s[3, [0, 2, 3]] == 0).all()
    assert y[4].isnan().all() and s[4].isnan().all()
    assert (y[5, :128] == 2).all() and (s[5, 1:] == 0).all() and (q[5, 128:] == 0).all() and (q[5, :128] == 0x7E).all()


# ------------------------------------------------------------------ grouped products

def make_groups(N, E, counts, R=0):
    """exp_off of the given rows an expert."""
    L = E // N
    c = torch.tensor(counts, dtype=torch.int64).view(N, L)
    off = torch.zeros((N, L + 1), dtype=torch.int64)
    off[:, 1:] = c.cumsum(1)
    return off.to(torch.int32).cuda()


def run_gemm(N, E, counts, K, F, T, k, R=0, swiglu=False, seed=1, spare=0):
    g = gen(seed)
    sh = moe.shape(N, T, 128, E, k, R)
    rows = moe.moe_recv_rows(sh)
    eo = make_groups(N, E, counts, R)
    x_q, x_s = X.quantise(torch.randn((rows, K), generator=g, device="cuda"))
    w_q, w_s = X.weights(E, 2 * F if swiglu else F, K, g)
    groups = X.group_rows(eo, rows, R)
    if swiglu:
        q = torch.full((rows, F), 0x5A, dtype=torch.uint8, device="cuda")
        s = torch.full((rows, F // 128), -3.0, device="cuda")
        moe.moe_grouped_gemm_swiglu(sh, x_q, x_s, w_q, w_s, eo, K, F, q, s)
    else:
        y = torch.full((rows, F), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_gemm(sh, x_q, x_s, w_q, w_s, eo, K, F, y)
    torch.cuda.synchronize()
    left = torch.ones(rows, dtype=torch.bool, device="cuda")
    if swiglu:
        for sl, a, da in X.swiglu(x_q, x_s, w_q, w_s, groups):
            X.check_quantised(q[sl], s[sl], a, da, f"rows {sl}")
            left[sl] = False
        assert (q[left] == 0x5A).all() and (s[left] == -3.0).all()
    else:
        for sl, r, d in X.gemm(x_q, x_s, w_q, w_s, groups):
            X.check_bf16(y[sl], r, d, f"rows {sl}")
            left[sl] = False
        assert (y[left] == 7.0).all()


def uneven(E, total, seed, zero_every=3):
    """Rows of E experts adding up to `total`, every third one without any."""
    g = torch.Generator().manual_seed(seed)
    p = torch.rand(E, generator=g) ** 2
    p[::zero_every] = 0 if E > 1 else 1
    c = (p / p.sum() * total).long()
    c[-1 if p[-1] > 0 else 1 if E > 1 else 0] += total - c.sum()
    return c.tolist()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N,E,T,k,K,F", [
    (1, 1, 1, 1, 128, 128),             # one row, one block
    (1, 1, 17, 1, 256, 256),
    (2, 8, 9, 2, 384, 256),             # a few rows an expert: the narrow tile
    (4, 16, 100, 4, 1024, 384),         # about 100: the middle tile
    (1, 2, 700, 2, 896, 256),           # many: the wide tile, 7 K steps
    (1, 1, 1337, 1, 1152, 128),         # 9 K steps
    (4, 1024, 5, 8, 256, 128),          # the most experts
    (1, 1, 257, 1, 2176, 640),          # one row over a tile, 17 K steps
    (2, 4, 513, 2, 2048, 384),          # 16 K steps
    (2, 8, 2000, 2, 384, 4096),         # enough tiles of 256 rows: the large tile
    (4, 512, 19200, 2, 128, 256),       # the same with more than 256 experts
])
def test_grouped_gemm_shapes(swiglu, N, E, T, k, K, F):
    log(f"gemm swiglu={swiglu} N={N} E={E} T={T} k={k} K={K} F={F}")
    run_gemm(N, E, uneven(E, N * T * k, T), K, F, T, k, swiglu=swiglu, seed=K)


@pytest.mark.parametrize("T,F", [(T, F) for T in (3, 90, 600) for F in (16, 48, 112, 144, 272, 400)] + [(8000, 4112)])
def test_grouped_gemm_odd_features(T, F):
    log(f"gemm F={F} T={T}")
    run_gemm(1, 2, [T - 1, T + 1], 384, F, T, 2, seed=F)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts", [[0, 0, 0, 600], [600, 0, 0, 0], [0, 0, 0, 0], [1, 1, 1, 1], [0, 32, 33, 31],
                                    [128, 127, 129, 1], [256, 255, 1, 0]])
def test_grouped_gemm_row_counts(swiglu, counts):
    log(f"gemm swiglu={swiglu} counts={counts}")
    for T in (150, 8):      # the shape's T chooses the tile; rows above what it allows are not made
        if sum(counts) <= 2 * T * 2:
            run_gemm(2, 4, counts, 256, 256, T, 2, swiglu=swiglu, seed=sum(counts))


@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_gemm_fixed_regions(swiglu):
    log(f"gemm fixed regions swiglu={swiglu}")
    run_gemm(2, 4, [10, 20, 0, 33], 256, 128, 40, 2, R=50, swiglu=swiglu)
    run_gemm(2, 4, [10, 60, 33, 40], 256, 128, 40, 2, R=50, swiglu=swiglu)     # both regions overflow
    run_gemm(2, 4, [70, 10, 0, 50], 256, 128, 40, 2, R=50, swiglu=swiglu)      # an expert past the region's end


def test_grouped_gemm_poisoned_neighbours():
    """Rows and experts that hold NaN leave every other row alone, and rows
    that no expert owns are not read into any."""
    g = gen(5)
    N, E, T, k, K, F = 1, 3, 40, 2, 256, 256
    sh = moe.shape(N, T, 128, E, k)
    eo = make_groups(N, E, [30, 20, 20])          # 10 rows behind the last
    x_q, x_s = X.quantise(torch.randn((80, K), generator=g, device="cuda"))
    w_q, w_s = X.weights(E, 2 * F, K, g)
    q, s = torch.empty((80, F), dtype=torch.uint8, device="cuda"), torch.zeros((80, 2), device="cuda")
    moe.moe_grouped_gemm_swiglu(sh, x_q, x_s, w_q, w_s, eo, K, F, q, s)
    q1, s1 = q.clone(), s.clone()
    x_q[70:] = 0x7F
    x_q[45] = 0x7F
    w_q[2] = 0x7F
    moe.moe_grouped_gemm_swiglu(sh, x_q, x_s, w_q, w_s, eo, K, F, q, s)
    keep = [i for i in range(50) if i != 45]
    assert torch.equal(q[keep], q1[keep]) and torch.equal(s[keep], s1[keep])
    assert s[45].isnan().all() and s[50:70].isnan().all()


def test_grouped_gemm_zero_rows_and_extremes():
    """A row of zeros gives zeros with scale 0; large scales reach infinity
    in bf16 only where the product does."""
    sh = moe.shape(1, 4, 128, 1, 1)
    eo = make_groups(1, 1, [4])
    g = gen(3)
    x_q, x_s = X.quantise(torch.randn((4, 256), generator=g, device="cuda"))
    x_q[1] = 0
    x_s[1] = 0
    x_s[2] *= 1e30
    w_q, w_s = X.weights(1, 256, 256, g)
    y = torch.empty((4, 256), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm(sh, x_q, x_s, w_q, w_s, eo, 256, 256, y)
    q, s = torch.empty((4, 128), dtype=torch.uint8, device="cuda"), torch.empty((4, 1), device="cuda")
    moe.moe_grouped_gemm_swiglu(sh, x_q, x_s, w_q, w_s, eo, 256, 128, q, s)
    assert (y[1] == 0).all() and (q[1] == 0).all() and s[1] == 0
    ref, d = X.product(X.values(x_q, x_s), X.values(w_q[0], w_s[0], 128), 256)
    X.check_bf16(y, ref, d + X._e4m3_products(X.values(x_q, x_s), X.values(w_q[0], w_s[0], 128)))


# ------------------------------------------------------------------ whole layer

def layer_inputs(N, T, H, E, k, I, seed=0):  # noqa: E741
    g = gen(seed)
    x = torch.randn((N, T, H), generator=g, device="cuda").bfloat16()
    v, i = torch.randn((N, T, E), generator=g, device="cuda").topk(k, 2)
    w13 = X.weights(E, 2 * I, H, g)
    w2 = X.weights(E, H, I, g)
    return x, i.int().contiguous(), torch.softmax(v, 2).contiguous(), *w13, *w2


def run_layer(N, T, H, E, k, I, x, idx, w, w13_q, w13_s, w2_q, w2_s):  # noqa: E741
    sh = moe.shape(N, T, H, E, k)
    ws = torch.full((moe.moe_layer_ll_workspace_bytes(sh, I),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(x, 9.0)
    flags = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    moe.moe_layer_ll(sh, x, idx, w, w13_q, w13_s, w2_q, w2_s, I, out, flags, ws)
    torch.cuda.synchronize()
    return out, int(flags.item())


def check_layer(out, N, T, H, k, x, idx, w, w13_q, w13_s, w2_q, w2_s):
    ref, bound = X.layer(x.view(-1, H), idx.view(-1, k), w.view(-1, k), w13_q, w13_s, w2_q, w2_s)
    X.check_bf16(out.view(-1, H), ref, bound, "out")


@pytest.mark.parametrize("N,T,H,E,k,I", [
    (1, 1, 128, 1, 1, 128),
    (1, 1, 2048, 16, 8, 512),
    (1, 1, 1152, 8, 1, 384),
    (2, 3, 640, 8, 2, 256),
    (1, 16, 512, 4, 2, 256),
    (1, 17, 512, 2, 1, 128),
    (4, 16, 256, 64, 8, 256),
    (8, 8, 384, 8, 8, 128),              # every token on every expert
    (64, 1, 256, 64, 1, 1152),
    (1, 64, 256, 1, 1, 640),
    (1, 3, 256, 1024, 64, 128),          # the most experts and slots a token
    (1, 40, 128, 3, 3, 128),             # 40 members an expert: four column tiles at once
    (1, 64, 384, 4, 1, 256),             # about 16: two tiles, with a second pass where there are more than 32
    (1, 48, 256, 24, 8, 256),            # 16 of 24 experts a token
])
def test_layer_shapes(N, T, H, E, k, I):  # noqa: E741
    log(f"layer N={N} T={T} H={H} E={E} k={k} I={I}")
    a = layer_inputs(N, T, H, E, k, I, seed=H + T)
    out, flags = run_layer(N, T, H, E, k, I, *a)
    assert flags == 0
    check_layer(out, N, T, H, k, *a)
    again, _ = run_layer(N, T, H, E, k, I, *a)
    assert torch.equal(out, again)


def test_layer_bad_repeated_and_missing_ids():
    N, T, H, E, k, I = 1, 6, 512, 8, 4, 256  # noqa: E741
    a = list(layer_inputs(N, T, H, E, k, I, seed=2))
    idx = a[1]
    idx[0, 0] = torch.tensor([3, 3, 5, 3])           # one expert three times
    idx[0, 1] = torch.tensor([-1, 8, 1 << 20, -(1 << 31)])   # none valid: a row of zeros
    idx[0, 2, 1] = 8
    idx[0, 3] = 7
    log("layer bad ids")
    out, flags = run_layer(N, T, H, E, k, I, *a)
    assert flags == moe.FLAG_BADID
    assert (out[0, 1] == 0).all()
    check_layer(out, N, T, H, k, *a)
    idx[:] = -5                                      # nothing valid at all
    out, flags = run_layer(N, T, H, E, k, I, *a)
    assert flags == moe.FLAG_BADID and (out == 0).all()
    idx[:] = 2                                       # one expert, every slot
    out, flags = run_layer(N, T, H, E, k, I, *a)
    assert flags == 0
    check_layer(out, N, T, H, k, *a)


def test_layer_nan_stays_with_its_token():
    N, T, H, E, k, I = 1, 20, 256, 4, 2, 256  # noqa: E741
    a = list(layer_inputs(N, T, H, E, k, I, seed=4))
    ref, _ = run_layer(N, T, H, E, k, I, *a)
    x = a[0].clone()
    x[0, 7, 3] = float("nan")
    x[0, 11, 5] = float("inf")
    out, _ = run_layer(N, T, H, E, k, I, x, *a[1:])
    keep = [t for t in range(T) if t not in (7, 11)]
    assert torch.equal(out[0, keep], ref[0, keep])
    assert out[0, 7].isnan().all() and not out[0, 11].isfinite().all()


def test_layer_in_place_and_empty():
    N, T, H, E, k, I = 1, 5, 256, 8, 2, 128  # noqa: E741
    a = layer_inputs(N, T, H, E, k, I, seed=6)
    ref, _ = run_layer(N, T, H, E, k, I, *a)
    sh = moe.shape(N, T, H, E, k)
    ws = torch.empty(moe.moe_layer_ll_workspace_bytes(sh, I), dtype=torch.uint8, device="cuda")
    flags = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    x = a[0].clone()
    moe.moe_layer_ll(sh, x, *a[1:], I, x, flags, ws)
    assert torch.equal(x, ref)
    flags.fill_(-1)
    moe.moe_layer_ll(moe.shape(2, 0, H, E, k), None, None, None, None, None, None, None, I, None, flags, None)
    assert int(flags.item()) == 0


# ------------------------------------------------------------------ together

def run_chain(cfg, I, R=0, direct=True):  # noqa: E741
    """norm -> dispatch -> gate/up product -> down product -> combine, plus a
    shared expert on the norm's own 8-bit rows; returns everything."""
    N, T, H, E, k = cfg.N, cfg.T, cfg.H, cfg.E, cfg.k
    g = gen(cfg.seed)
    c = dict(sh=moe.shape(N, T, H, E, k, R), shared=moe.shape(1, N * T, H, 1, 1))
    idx, w = W.routing(cfg)
    c["idx"], c["w"] = torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda()
    c["x"], c["res"] = (torch.randn((N, T, H), generator=g, device="cuda").bfloat16() for _ in range(2))
    c["gamma"] = torch.randn(H, generator=g, device="cuda").abs().bfloat16()
    c["w13"], c["w2"] = X.weights(E, 2 * I, H, g), X.weights(E, H, I, g)
    c["s13"], c["s2"] = X.weights(1, 2 * I, H, g), X.weights(1, H, I, g)
    B = c["B"] = moe.allocate(c["sh"], "cuda")
    rows = B.rows
    c["res_out"], c["y"] = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    c["y_q"] = torch.empty((N * T, H), dtype=torch.uint8, device="cuda")
    c["y_s"] = torch.empty((N * T, H // 128), device="cuda")
    c["a_q"], c["a_s"] = torch.empty((rows, I), dtype=torch.uint8, device="cuda"), torch.empty((rows, I // 128), device="cuda")
    c["sa_q"], c["sa_s"] = torch.empty((N * T, I), dtype=torch.uint8, device="cuda"), torch.empty((N * T, I // 128), device="cuda")
    c["y_em"] = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    c["s_out"] = torch.empty((N * T, H), dtype=torch.bfloat16, device="cuda")
    c["one"] = torch.tensor([[0, N * T]], dtype=torch.int32, device="cuda")

    def go():
        moe.moe_rmsnorm_quant(c["sh"], c["x"], c["res"], c["gamma"], 1e-6, c["res_out"], c["y"], c["y_q"], c["y_s"])
        moe.moe_dispatch_direct(c["sh"], c["y"], c["idx"], B.x_q, B.x_s, B.send_pos, B.exp_off, B.row_src, B.ws)
        moe.moe_grouped_gemm_swiglu(c["sh"], B.x_q, B.x_s, *c["w13"], B.exp_off, H, I, c["a_q"], c["a_s"])
        moe.moe_grouped_gemm(c["sh"], c["a_q"], c["a_s"], *c["w2"], B.exp_off, I, H, c["y_em"])
        moe.moe_combine_pull(c["sh"], c["y_em"], c["idx"], B.send_pos, c["w"], B.ws, B.out)
        moe.moe_grouped_gemm_swiglu(c["shared"], c["y_q"], c["y_s"], *c["s13"], c["one"], H, I, c["sa_q"], c["sa_s"])
        moe.moe_grouped_gemm(c["shared"], c["sa_q"], c["sa_s"], *c["s2"], c["one"], I, H, c["s_out"])
    c["go"] = go
    return c


CHAIN = W.Config("chain", N=4, T=50, H=512, E=16, k=4, seed=77)


@pytest.mark.parametrize("R", [0, 4 * 50 * 4])
def test_chain(R):
    log(f"chain R={R}")
    I = 256  # noqa: E741
    c = run_chain(CHAIN, I, R)
    c["go"]()
    B, rows = c["B"], c["B"].rows
    assert moe.moe_status(B.ws) == 0
    groups = X.group_rows(B.exp_off, rows, R)
    assert sum(n for _, _, n in groups) == CHAIN.N * CHAIN.T * CHAIN.k
    for sl, a, da in X.swiglu(B.x_q, B.x_s, *c["w13"], groups):
        X.check_quantised(c["a_q"][sl], c["a_s"][sl], a, da)
    for sl, y, d in X.gemm(c["a_q"], c["a_s"], *c["w2"], groups):
        X.check_bf16(c["y_em"][sl], y, d)
    for sl, a, da in X.swiglu(c["y_q"], c["y_s"], *c["s13"], [(0, 0, CHAIN.N * CHAIN.T)]):
        X.check_quantised(c["sa_q"][sl], c["sa_s"][sl], a, da)
    for sl, y, d in X.gemm(c["sa_q"], c["sa_s"], *c["s2"], [(0, 0, CHAIN.N * CHAIN.T)]):
        X.check_bf16(c["s_out"][sl], y, d)
    # the combined layer against the layer on unquantised tokens: the three 8-bit roundings
    # (tokens and activation, each half a step) are 2^-4 each at the worst, far less in the norm
    ref, _ = X.layer(c["y"].view(-1, CHAIN.H), c["idx"].view(-1, CHAIN.k), c["w"].view(-1, CHAIN.k), *c["w13"], *c["w2"])
    off = (B.out.view(-1, CHAIN.H).double() - ref).norm() / ref.norm()
    assert off < 2 * 2.0 ** -4


def test_chain_and_layer_agree():
    """The same tokens through dispatch and through the few-token layer."""
    cfg = W.Config("chain64", N=4, T=16, H=512, E=16, k=4, seed=78)
    c = run_chain(cfg, 256)
    c["go"]()
    out, flags = run_layer(4, 16, 512, 16, 4, 256, c["y"], c["idx"], c["w"], *c["w13"], *c["w2"])
    assert flags == 0
    off = (out.double() - c["B"].out.double()).norm() / out.double().norm()
    assert off < 2 * 2.0 ** -4


def test_chain_in_a_graph_and_on_another_stream():
    """Captured, replayed with new inputs and eager work between the replays;
    then on a stream that is not the current one."""
    log("chain in a graph")
    c = run_chain(CHAIN, 256)
    B = c["B"]
    N, T, H, E, k = CHAIN.N, 2, CHAIN.H, CHAIN.E, CHAIN.k
    sh = moe.shape(N, T, H, E, k)
    ws = torch.empty(moe.moe_layer_ll_workspace_bytes(sh, 256), dtype=torch.uint8, device="cuda")
    lx, lidx, lw = c["x"][:, :T].contiguous(), c["idx"][:, :T].contiguous(), c["w"][:, :T].contiguous()
    lout, flags = torch.empty_like(lx), torch.empty(1, dtype=torch.int32, device="cuda")

    def go():
        c["go"]()
        moe.moe_layer_ll(sh, lx, lidx, lw, *c["w13"], *c["w2"], 256, lout, flags, ws)
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    outs = (B.out, c["s_out"], c["res_out"], lout)
    g = gen(9)
    for _ in range(3):
        c["x"].copy_(torch.randn(c["x"].shape, generator=g, device="cuda"))
        lx.copy_(c["x"][:, :T])
        go()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, v in zip(outs, want):
            assert torch.equal(t, v)
    side = torch.cuda.Stream()
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    for t, v in zip(outs, want):
        assert torch.equal(t, v)


# ------------------------------------------------------------------ large offsets

def test_grouped_gemm_offsets_beyond_32_bits():
    """Rows and weights behind the first 2^31 bytes: the ends of the arrays
    against a plain product."""
    g = gen(31)
    T, K, F = 153000, 7168, 128                       # 306000 rows of 7168 bytes
    sh = moe.shape(1, T, 128, 2, 2)
    rows = moe.moe_recv_rows(sh)
    log(f"gemm rows={rows} K={K} F={F}")
    eo = make_groups(1, 2, [rows - 70, 70])
    x_q = torch.randint(0, 0x70, (rows, K), dtype=torch.uint8, generator=g, device="cuda")
    x_s = torch.rand((rows, K // 128), generator=g, device="cuda")
    w_q, w_s = X.weights(2, F, K, g)
    y = torch.empty((rows, F), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm(sh, x_q, x_s, w_q, w_s, eo, K, F, y)
    groups = [(0, 0, 40), (0, rows - 110, 40), (1, rows - 70, 70)]
    for sl, r, d in X.gemm(x_q, x_s, w_q, w_s, groups):
        X.check_bf16(y[sl], r, d, str(sl))
    del x_q, x_s, y
    E, F, T = 40, 8192, 20                             # 2.35 GB of weights
    log(f"gemm E={E} F={F} K={K}")
    sh = moe.shape(1, T, 128, E, 2)
    counts = [0] * E
    counts[0], counts[E - 1] = 3, 37
    eo = make_groups(1, E, counts)
    x_q, x_s = X.quantise(torch.randn((40, K), generator=g, device="cuda"))
    w_q = torch.randint(0, 0x70, (E, F, K), dtype=torch.uint8, generator=g, device="cuda")
    w_s = torch.rand((E, F // 128, K // 128), generator=g, device="cuda") * 1e-3
    y = torch.empty((40, F), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm(sh, x_q, x_s, w_q, w_s, eo, K, F, y)
    for sl, r, d in X.gemm(x_q, x_s, w_q, w_s, [(0, 0, 3), (E - 1, 3, 37)]):
        X.check_bf16(y[sl], r, d, str(sl))
    q, s = torch.empty((40, F // 2), dtype=torch.uint8, device="cuda"), torch.empty((40, F // 256), device="cuda")
    moe.moe_grouped_gemm_swiglu(sh, x_q, x_s, w_q, w_s, eo, K, F // 2, q, s)
    for sl, a, da in X.swiglu(x_q, x_s, w_q, w_s, [(0, 0, 3), (E - 1, 3, 37)]):
        X.check_quantised(q[sl], s[sl], a, da, str(sl))


def test_layer_weights_beyond_32_bits():
    N, T, H, E, k, I = 1, 3, 7168, 64, 2, 2560  # noqa: E741   2.35 GB of gate/up weights
    log(f"layer E={E} H={H} I={I}")
    g = gen(8)
    x = torch.randn((N, T, H), generator=g, device="cuda").bfloat16()
    idx = torch.tensor([[[E - 1, 0], [E - 2, E - 1], [1, E - 3]]], dtype=torch.int32, device="cuda")
    w = torch.rand((N, T, k), generator=g, device="cuda")
    f8 = lambda *s: torch.randint(0, 0x68, s, dtype=torch.uint8, generator=g, device="cuda")  # noqa: E731
    w13_q, w2_q = f8(E, 2 * I, H) ^ (f8(E, 2 * I, H) & 1) << 7, f8(E, H, I) ^ (f8(E, H, I) & 1) << 7
    w13_s = torch.rand((E, 2 * I // 128, H // 128), generator=g, device="cuda") * 1e-3
    w2_s = torch.rand((E, H // 128, I // 128), generator=g, device="cuda") * 1e-3
    a = (x, idx, w, w13_q, w13_s, w2_q, w2_s)
    out, flags = run_layer(N, T, H, E, k, I, *a)
    assert flags == 0
    check_layer(out, N, T, H, k, *a)


def test_norm_rows_beyond_32_bits():
    T, H = 300000, 7168                               # 2.15e9 elements
    log(f"norm T={T} H={H}")
    g = gen(4)
    sh = moe.shape(1, T, H, 1, 1)
    x = torch.randn((1, T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    gamma = torch.randn(H, generator=g, device="cuda").bfloat16()
    y = torch.empty_like(x)
    q, s = torch.empty((1, T, H), dtype=torch.uint8, device="cuda"), torch.empty((1, T, H // 128), device="cuda")
    moe.moe_rmsnorm_quant(sh, x, None, gamma, 1e-6, None, y, q, s)
    for sl in (slice(0, 20), slice(T - 20, T)):
        _, n, rel = X.norm(x[0, sl], None, gamma, 1e-6)
        X.check_bf16(y[0, sl], n, n.abs() * rel)
        X.check_quantised(q[0, sl], s[0, sl], n, n.abs() * rel)


def test_norm_more_rows_than_one_launch():
    """Above 2^21 rows the call takes several launches."""
    T, H = (1 << 21) + 3, 128
    log(f"norm T={T} H={H}")
    g = gen(6)
    sh = moe.shape(1, T, H, 1, 1)
    x, res = (torch.randn((1, T, H), generator=g, device="cuda").bfloat16() for _ in range(2))
    gamma = torch.randn(H, generator=g, device="cuda").bfloat16()
    r, y = torch.empty_like(x), torch.empty_like(x)
    q, s = torch.empty((1, T, H), dtype=torch.uint8, device="cuda"), torch.empty((1, T, 1), device="cuda")
    moe.moe_rmsnorm_quant(sh, x, res, gamma, 1e-6, r, y, q, s)
    for sl in (slice(0, 9), slice((1 << 21) - 5, T)):
        ref, n, rel = X.norm(x[0, sl], res[0, sl], gamma, 1e-6)
        X.check_bf16(r[0, sl], ref, ref.abs() * X.U)
        X.check_bf16(y[0, sl], n, n.abs() * rel)
        X.check_quantised(q[0, sl], s[0, sl], n, n.abs() * rel)
