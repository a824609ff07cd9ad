"""The operators that train an expert layer, on the GPU against plain float64
forms (tests/training_ref.py), at the sizes, layouts and values where they can
go wrong, and a run of them together as a layer, forwards and backwards."""
import pytest
import torch

import combine_lds_atomic_amd as moe
import expert_ref as X
import training_ref as R

pytestmark = pytest.mark.gpu

from gpu_harness import log  # noqa: E402

BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def make_groups(N, E, counts):
    """exp_off of the given rows an expert."""
    c = torch.tensor(counts, dtype=torch.int64).view(N, E // N)
    off = torch.zeros((N, E // N + 1), dtype=torch.int64)
    off[:, 1:] = c.cumsum(1)
    return off.to(torch.int32).cuda()


def uneven(E, total, seed, zero_every=3):
    """Rows of E experts adding up to `total`, every third one without any."""
    g = torch.Generator().manual_seed(seed)
    p = torch.rand(E, generator=g) ** 2
    p[::zero_every] = 0 if E > 1 else 1
    c = (p / p.sum() * total).long()
    c[-1 if p[-1] > 0 else 1 if E > 1 else 0] += total - c.sum()
    return c.tolist()


# ------------------------------------------------------------------ products

def run_products(N, E, counts, H, I, T, k, R_=0, seed=1, flags=True):  # noqa: E741
    """Every product call on one load: up, the down product, up's gradient, the
    rows' and the weights' gradients, each against its own inputs."""
    g = gen(seed)
    sh = moe.shape(N, T, 128, E, k, R_)
    rows = moe.moe_recv_rows(sh)
    eo = make_groups(N, E, counts)
    groups = X.group_rows(eo, rows, R_)
    x, dy = normal((rows, H), g), normal((rows, H), g)
    w13, w2 = normal((E, 2 * I, H), g, H ** -0.5), normal((E, H, I), g, I ** -0.5)
    new = lambda *s: torch.full(s, 7.0, dtype=BF, device="cuda")  # noqa: E731
    a, y, dh, a2, dx = new(rows, I), new(rows, H), new(rows, 2 * I), new(rows, I), new(rows, H)
    h_q = torch.full((rows, 2 * I), 0x5A, dtype=torch.uint8, device="cuda")
    h_s = torch.full((rows, 2 * I // 128), -3.0, device="cuda")
    moe.moe_ffn_up(sh, x, w13, eo, H, I, a, h_q, h_s)
    moe.moe_grouped_gemm_bf16(sh, a, w2, eo, I, H, False, y)
    moe.moe_ffn_up_grad(sh, dy, w2, h_q, h_s, eo, H, I, dh, a2)
    moe.moe_grouped_gemm_bf16(sh, dh, w13, eo, 2 * I, H, True, dx)
    dw = {(t, add): torch.ones((E, 2 * I, H), dtype=t, device="cuda") for t in (BF, torch.float32)
          for add in (False, True)}
    dw2 = torch.empty((E, H, I), dtype=BF, device="cuda")
    for (_, add), v in dw.items():
        moe.moe_grouped_wgrad(sh, dh, x, eo, 2 * I, H, v, add)
    moe.moe_grouped_wgrad(sh, dy, a2, eo, H, I, dw2)
    torch.cuda.synchronize()
    left = torch.ones(rows, dtype=torch.bool, device="cuda")
    for e, first, n in groups:
        sl = slice(first, first + n)
        left[sl] = False
        if n:
            av, ab, hv, hb = R.up(x[sl], w13[e])
            X.check_bf16(a[sl], av, ab, f"a of expert {e}")
            X.check_quantised(h_q[sl], h_s[sl], hv, hb, f"h of expert {e}")
            X.check_bf16(y[sl], *R.product(a[sl], w2[e]), f"y of expert {e}")
            hv, hb, av, ab = R.up_grad(dy[sl], w2[e], h_q[sl], h_s[sl])
            X.check_bf16(dh[sl], hv, hb, f"dh of expert {e}")
            X.check_bf16(a2[sl], av, ab, f"a again of expert {e}")
            X.check_bf16(dx[sl], *R.product(dh[sl], w13[e], True), f"dx of expert {e}")
        if not n:
            assert (dw2[e] == 0).all() and all((v[e] == add).all() for (_, add), v in dw.items()), f"empty expert {e}"
            continue
        v, b = R.wgrad(dh[sl], x[sl])
        X.check_bf16(dw[BF, False][e], v, b, f"dw13 of expert {e}")
        R.check_f32(dw[torch.float32, False][e], v, b, f"dw13 in fp32 of expert {e}")
        X.check_bf16(dw[BF, True][e], v + 1, b + (v + 1).abs() * R.U, f"dw13 added of expert {e}")
        R.check_f32(dw[torch.float32, True][e], v + 1, b, f"dw13 added in fp32 of expert {e}")
        X.check_bf16(dw2[e], *R.wgrad(dy[sl], a2[sl]), f"dw2 of expert {e}")
    for t, old in ((a, 7.0), (y, 7.0), (dh, 7.0), (a2, 7.0), (dx, 7.0), (h_q, 0x5A), (h_s, -3.0)):
        assert (t[left] == old).all()


@pytest.mark.parametrize("N,E,T,k,H,I", [
    (1, 1, 1, 1, 128, 128),             # one row, one block
    (1, 1, 17, 1, 256, 256),
    (2, 8, 9, 2, 384, 256),             # a few rows an expert: the narrow tile
    (4, 16, 100, 4, 1024, 384),         # about 100: the middle tile
    (1, 2, 700, 2, 896, 256),           # several tiles, 14 K steps
    (1, 1, 1337, 1, 1152, 128),         # 18 K steps
    (4, 1024, 5, 8, 256, 128),          # the most experts
    (1, 1, 257, 1, 2176, 640),          # one row over a tile, 34 K steps
    (2, 4, 513, 2, 2048, 384),
    (2, 8, 2000, 2, 384, 4096),         # enough tiles of 256 rows: the large tile
    (1, 320, 3000, 1, 128, 128),        # more than 256 experts, uneven
    (4, 64, 400, 4, 1024, 640),         # the middle tile on every side
    (1, 320, 30000, 1, 128, 128),       # the same with more than 256 experts
    (2, 32, 2500, 2, 2048, 256),        # the large tile for the products of rows and of columns
    (2, 32, 2500, 2, 256, 2048),        # and for the up product's gradient
    (4, 512, 25600, 1, 128, 128),       # the same with more than 256 experts
    (1, 1, 1337, 1, 6912, 256),         # one expert in one round of large tiles
    (1, 1, 2300, 1, 256, 2048),         # and its up product
])
def test_products_shapes(N, E, T, k, H, I):  # noqa: E741
    log(f"products N={N} E={E} T={T} k={k} H={H} I={I}")
    run_products(N, E, uneven(E, N * T * k, T), H, I, T, k, seed=H)


@pytest.mark.parametrize("counts", [[0, 0, 0, 600], [600, 0, 0, 0], [0, 0, 0, 0], [1, 1, 1, 1], [0, 32, 33, 31],
                                    [128, 127, 129, 1], [256, 255, 1, 0], [64, 65, 63, 2]])
def test_products_row_counts(counts):
    log(f"products counts={counts}")
    for T in (150, 8):      # the shape's T chooses the tile; rows above what it allows are not made
        if sum(counts) <= 2 * T * 2:
            run_products(2, 4, counts, 256, 128, T, 2, seed=sum(counts))


def test_products_fixed_regions():
    log("products fixed regions")
    run_products(2, 4, [10, 20, 0, 33], 256, 128, 40, 2, R_=50)
    run_products(2, 4, [10, 60, 33, 40], 256, 128, 40, 2, R_=50)     # both regions overflow
    run_products(2, 4, [70, 10, 0, 50], 256, 128, 40, 2, R_=50)      # an expert past the region's end


@pytest.mark.parametrize("F", [16, 48, 112, 144, 272, 400, 4112])
@pytest.mark.parametrize("T", [3, 90, 600])
def test_gemm_and_wgrad_odd_features(T, F):
    """Features that end inside a tile, on either side of a product."""
    log(f"odd features F={F} T={T}")
    g, E, K = gen(F + T), 2, 384
    sh = moe.shape(1, T, 128, E, 2)
    eo = make_groups(1, E, [T - 1, T + 1])
    x, d = normal((2 * T, K), g), normal((2 * T, F), g)
    w = normal((E, F, K), g, K ** -0.5)
    wt = w.transpose(1, 2).contiguous()
    y, yt = (torch.empty((2 * T, F), dtype=BF, device="cuda") for _ in range(2))
    dw, dwt = torch.empty((E, F, K), device="cuda"), torch.empty((E, K, F), device="cuda")
    moe.moe_grouped_gemm_bf16(sh, x, w, eo, K, F, False, y)
    moe.moe_grouped_gemm_bf16(sh, x, wt, eo, K, F, True, yt)
    moe.moe_grouped_wgrad(sh, d, x, eo, F, K, dw)
    moe.moe_grouped_wgrad(sh, x, d, eo, K, F, dwt)
    for e, a, n in X.group_rows(eo, 2 * T, 0):
        sl = slice(a, a + n)
        for got in (y, yt):
            X.check_bf16(got[sl], *R.product(x[sl], w[e]), f"expert {e}")
        v, b = R.wgrad(d[sl], x[sl])
        R.check_f32(dw[e], v, b, f"dw of expert {e}")
        R.check_f32(dwt[e], v.T, b.T, f"dw the other way of expert {e}")


def test_products_poisoned_neighbours():
    """Rows and experts that hold NaN or infinities leave every other row and
    expert alone, and rows that no expert owns are not read into any."""
    g, N, E, T, k, H, I = gen(5), 1, 3, 40, 2, 256, 256  # noqa: E741
    sh = moe.shape(N, T, 128, E, k)
    eo = make_groups(N, E, [30, 20, 20])          # 10 rows behind the last
    x, dy = normal((80, H), g), normal((80, H), g)
    w13, w2 = normal((E, 2 * I, H), g, 0.06), normal((E, H, I), g, 0.06)

    def step():
        a, y = torch.zeros((80, I), dtype=BF, device="cuda"), torch.zeros((80, H), dtype=BF, device="cuda")
        q, s = torch.zeros((80, 2 * I), dtype=torch.uint8, device="cuda"), torch.zeros((80, 4), device="cuda")
        dh, dx, a2 = torch.zeros((80, 2 * I), dtype=BF, device="cuda"), torch.zeros_like(y), torch.zeros_like(a)
        dw13, dw2 = torch.zeros((E, 2 * I, H), device="cuda"), torch.zeros((E, H, I), device="cuda")
        moe.moe_ffn_up(sh, x, w13, eo, H, I, a, q, s)
        moe.moe_grouped_gemm_bf16(sh, a, w2, eo, I, H, False, y)
        moe.moe_ffn_up_grad(sh, dy, w2, q, s, eo, H, I, dh, a2)
        moe.moe_grouped_gemm_bf16(sh, dh, w13, eo, 2 * I, H, True, dx)
        moe.moe_grouped_wgrad(sh, dh, x, eo, 2 * I, H, dw13)
        moe.moe_grouped_wgrad(sh, dy, a2, eo, H, I, dw2)
        return a, y, q, s, dh, dx, dw13, dw2
    first = step()
    x[70:], dy[70:] = float("nan"), float("inf")
    assert all(torch.equal(u, v) for u, v in zip(first, step()))
    x[45] = float("nan")                          # expert 1
    w13[2], w2[2] = float("inf"), float("nan")
    again = step()
    ok = torch.ones(70, dtype=torch.bool, device="cuda")
    ok[45] = ok[50:] = False
    for u, v in zip(first[:6], again[:6]):
        assert torch.equal(u[:70][ok], v[:70][ok])
    assert torch.equal(first[6][0], again[6][0]) and torch.equal(first[7][0], again[7][0])
    assert again[1][45].isnan().all() and again[6][1].isnan().any() and again[0][50:70].isnan().any()


def test_up_values():
    """Gates far from zero: silu and its gradient saturate without NaN."""
    log("up values")
    H, I = 128, 128  # noqa: E741
    sh = moe.shape(1, 4, 128, 1, 1)
    eo = make_groups(1, 1, [4])
    x = torch.zeros((4, H), dtype=BF, device="cuda")
    x[:, 0] = torch.tensor([1e4, -1e4, 0.0, 1e-20], device="cuda").to(BF)
    w13 = torch.ones((1, 2 * I, H), dtype=BF, device="cuda")
    w2 = torch.ones((1, H, I), dtype=BF, device="cuda")
    dy = torch.ones((4, H), dtype=BF, device="cuda")
    a, dh, a2 = (torch.empty((4, n), dtype=BF, device="cuda") for n in (I, 2 * I, I))
    q, s = torch.empty((4, 2 * I), dtype=torch.uint8, device="cuda"), torch.empty((4, 2), device="cuda")
    moe.moe_ffn_up(sh, x, w13, eo, H, I, a, q, s)
    moe.moe_ffn_up_grad(sh, dy, w2, q, s, eo, H, I, dh, a2)
    big = float(torch.tensor(1e4).to(BF))
    assert torch.allclose(a[0].float(), torch.tensor(big * big, device="cuda"), rtol=2.0 ** -7)
    assert (a[1:3] == 0).all() and (a2[1:3] == 0).all()
    assert torch.allclose(dh[0].float(), torch.tensor(128 * big, device="cuda"), rtol=2.0 ** -7)
    assert (dh[1:3] == 0).all() and (q[2] == 0).all() and (s[2] == 0).all()
    assert dh.isfinite().all() and a.isfinite().all()
    none = torch.empty_like(a)
    moe.moe_ffn_up(sh, x, w13, eo, H, I, none, None, None)         # no checkpoint: the same rows
    assert torch.equal(a, none)
    dh2 = torch.empty_like(dh)
    moe.moe_ffn_up_grad(sh, dy, w2, q, s, eo, H, I, dh2, None)
    assert torch.equal(dh, dh2)


def test_products_offsets_beyond_32_bits():
    """Rows, weights and outputs more than 2^31 elements (and 2^32 bytes) from
    their arrays' starts."""
    log("offsets beyond 32 bits")
    g, E, H, I = gen(3), 3, 32768, 32768  # noqa: E741
    sh = moe.shape(1, 70000, 128, E, 1)
    eo = make_groups(1, E, [69990, 0, 10])
    w = torch.zeros((E, H, I), dtype=BF, device="cuda")
    w[2] = normal((H, I), g, I ** -0.5)
    x = torch.zeros((70000, I), dtype=BF, device="cuda")
    x[69990:] = normal((10, I), g)
    y = torch.zeros((70000, H), dtype=BF, device="cuda")
    for w_t in (False, True):
        moe.moe_grouped_gemm_bf16(sh, x, w, eo, I, H, w_t, y)
        X.check_bf16(y[69990:], *R.product(x[69990:], w[2], w_t), "y")
        assert (y[:69990] == 0).all()
    moe.moe_grouped_wgrad(sh, y, x, eo, H, I, w)
    X.check_bf16(w[2], *R.wgrad(y[69990:], x[69990:]), "dw")
    assert (w[:2] == 0).all()


def test_up_largest_features():
    """The largest K and I: an expert's up rows lie 2^31 bytes behind its gate rows."""
    log("up, largest features")
    g, n, K = gen(11), 5, 32768
    sh, eo = moe.shape(1, n, 128, 1, 1), make_groups(1, 1, [n])
    w13 = torch.zeros((1, 2 * K, K), dtype=BF, device="cuda")
    for f in (0, K - 128, K, 2 * K - 128):
        w13[0, f:f + 128] = normal((128, K), g, K ** -0.5)
    x = normal((n, K), g)
    a = torch.empty((n, K), dtype=BF, device="cuda")
    q, s = torch.empty((n, 2 * K), dtype=torch.uint8, device="cuda"), torch.empty((n, 2 * K // 128), device="cuda")
    moe.moe_ffn_up(sh, x, w13, eo, K, K, a, q, s)
    for f in (0, K - 128):
        part = torch.cat((w13[0, f:f + 128], w13[0, K + f:K + f + 128]))
        av, ab, hv, hb = R.up(x, part)
        R.check_bf16(a[:, f:f + 128], av, ab, f"a from {f}")
        for half in (0, 1):
            c = slice(half * K + f, half * K + f + 128)
            h = slice(half * 128, half * 128 + 128)
            X.check_quantised(q[:, c].contiguous(), s[:, c.start // 128:c.start // 128 + 1], hv[:, h], hb[:, h])
    assert (a[:, 128:K - 128] == 0).all()


# ------------------------------------------------------------------ combine

def routed(N, T, E, k, H, seed, R_=0, bad=False, early=0):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(N * T)]).view(N, T, k).to(torch.int32)
    if bad:
        idx[0, 0, 0] = E
        idx[-1, -1, -1] = -1
        if k > 1:
            idx[0, T // 2, 1] = idx[0, T // 2, 0]       # the same expert twice
    w = torch.softmax(torch.randn((N, T, k), generator=g), -1)
    sh = moe.shape(N, T, H, E, k, R_, early)
    B = moe.allocate(sh, "cuda", payload=False, combine=False)
    idx = idx.cuda()
    moe.moe_dispatch_direct(sh, None, idx, None, None, B.send_pos, B.exp_off, B.row_src, B.ws)
    return sh, B, idx, w.cuda()


def slot_rows(sh, B):
    """Row of every slot [N, T, k], -1 for none, from row_src and send_pos."""
    tk = sh.T * sh.k
    of = torch.full((sh.N * tk + 1,), -1, dtype=torch.int64, device="cuda")
    base = 0
    for d, n in enumerate(B.exp_off[:, -1].tolist()):
        start = d * sh.region_rows if sh.region_rows else base
        n = min(n, sh.region_rows) if sh.region_rows else n
        src = B.row_src[start:start + n].long()
        of[src] = torch.arange(start, start + n, device="cuda")      # -1 lands on the spare last place
        base += n
    of[-1] = -1
    pos = B.send_pos.long()
    at = pos + torch.arange(sh.N, device="cuda")[:, None, None] * tk
    return torch.where(pos >= 0, of[at.clamp(min=0)], -1)


@pytest.mark.parametrize("N,T,E,k,H,R_,bad,early", [
    (1, 1, 1, 1, 128, 0, False, 0),
    (1, 3, 8, 5, 384, 0, False, 0),
    (4, 50, 16, 4, 1024, 0, True, 0),
    (2, 700, 8, 8, 2048, 0, False, 0),
    (2, 9, 64, 64, 640, 0, False, 0),            # the most slots a token
    (8, 33, 32, 6, 7168, 0, True, 0),
    (2, 5, 4, 3, 8192, 0, False, 0),
    (2, 5, 4, 3, 8320, 0, False, 0),             # more than a wave holds at once
    (1, 7, 4, 2, 32768, 0, False, 0),
    (4, 50, 16, 4, 256, 400, True, 0),           # fixed regions, all rows fit
    (4, 50, 16, 4, 256, 150, True, 0),           # overflowing
    (4, 50, 16, 4, 256, 200, False, 45),         # with early rows: rows without a token in between
])
def test_combine_grad(N, T, E, k, H, R_, bad, early):
    log(f"combine grad N={N} T={T} E={E} k={k} H={H} R={R_} bad={bad} early={early}")
    sh, B, idx, w = routed(N, T, E, k, H, T, R_, bad, early)
    g = gen(T)
    rows = moe.moe_recv_rows(sh)
    dout, y = normal((N, T, H), g), normal((rows, H), g)
    dy, dw = torch.full((rows, H), 7.0, dtype=BF, device="cuda"), torch.full((N, T, k), 9.0, device="cuda")
    moe.moe_combine_grad(sh, dout, y, idx, B.send_pos, w, B.row_src, B.ws, dy, dw)
    at = slot_rows(sh, B)
    has = at >= 0
    want = dout.double()[:, :, None] * w.double()[..., None]
    terms = dout.double()[:, :, None] * y.double()[at.clamp(min=0)]
    X.check_bf16(dy[at[has]], want[has], want[has].abs() * R.U, "dy")
    R.check_f32(dw[has], terms.sum(-1)[has], (terms.abs().sum(-1) * (H / 64 + 16) * R.U)[has], "dw")
    assert (dw[~has] == 0).all()
    other = torch.ones(rows, dtype=torch.bool, device="cuda")
    other[at[has]] = False
    if R_:
        start = 0
        for d, n in enumerate(B.exp_off[:, -1].tolist()):
            sl = slice(d * R_, d * R_ + min(n, R_))
            assert (dy[sl][other[sl]] == 0).all()        # rows that an overflow left without a token
            other[sl] = False
            start += n
    assert (dy[other] == 7.0).all()
    # the choice of outputs changes none of them; dy over y
    dy2, dw2 = torch.full_like(dy, 7.0), torch.empty_like(dw)
    moe.moe_combine_grad(sh, dout, None, idx, B.send_pos, w, B.row_src, B.ws, dy2, None)
    moe.moe_combine_grad(sh, dout, y, idx, B.send_pos, w, B.row_src, B.ws, None, dw2)
    assert torch.equal(dy, dy2) and torch.equal(dw, dw2)
    keep = y.clone()
    moe.moe_combine_grad(sh, dout, y, idx, B.send_pos, w, B.row_src, B.ws, y, dw2)
    assert torch.equal(dw, dw2) and torch.equal(y[at[has]], dy[at[has]])
    if not R_:
        assert torch.equal(y[other], keep[other])
    # without weights: the tokens' rows, which the pulling combine brings back
    moe.moe_combine_grad(sh, dout, None, idx, B.send_pos, None, B.row_src, B.ws, dy2, None)
    assert torch.equal(dy2[at[has]], dout[:, :, None].expand(N, T, k, H)[has])


# ------------------------------------------------------------------ norms around a block

def norm_case(N, T, H, seed):
    g = gen(seed)
    r = lambda std=1.0: normal((N, T, H), g, std)  # noqa: E731
    gp, gn = ((1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF) for _ in range(2))
    gate = torch.randn((N, T), generator=g, device="cuda")
    return moe.shape(N, T, H, N, 1), r(0.3), r(4.0), gp, gate, gn, r(), r()


def check_norm(sh, x, res, gp, gate, alpha, gn, eps=1e-5):
    r_out, y = torch.empty_like(x), torch.empty_like(x) if gn is not None else None
    moe.moe_block_norm(sh, x, res, gp, gate, alpha, gn, eps, r_out, y)
    r, br, yv, by = R.block_norm(x, res, gp, gate, alpha, gn, eps)
    X.check_bf16(r_out, r, br, "r")
    if gn is not None:
        X.check_bf16(y, yv, by, "y")
    return r_out, y


def check_norm_grad(sh, dy, dr, x, res, gp, gate, alpha, gn, eps=1e-5):
    new = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    got = {"dx": torch.empty_like(x), "dresidual": torch.empty_like(x), "dgate": new(sh.N, sh.T),
           "dgamma_post": new(sh.H), "dgamma_next": new(sh.H) if gn is not None else None}
    ws = torch.empty(moe.moe_block_norm_grad_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    moe.moe_block_norm_grad(sh, dy, dr, x, res, gp, gate, alpha, gn, eps, *got.values(), ws)
    for n, (v, b) in R.block_norm_grad(dy, dr, x, res, gp, gate, alpha, gn, eps).items():
        (R.check_bf16 if n in ("dx", "dresidual") else R.check_f32)(got[n], v, b, n)
    return got


@pytest.mark.parametrize("H", [128, 384, 512, 640, 1024, 1152, 2048, 7168, 8192, 8320, 16384, 20480, 32768])
@pytest.mark.parametrize("T", [1, 5])
def test_block_norm_sizes(H, T):
    log(f"block norm H={H} T={T}")
    sh, x, res, gp, gate, gn, dy, dr = norm_case(1, T, H, H + T)
    check_norm(sh, x, res, gp, gate, 0.75, gn)
    check_norm_grad(sh, dy, dr, x, res, gp, gate, 0.75, gn)


@pytest.mark.parametrize("N,T,H", [(3, 7, 256), (2, 3000, 1024), (8, 33, 7168), (3, 5001, 128)])
def test_block_norm_many_rows_and_in_place(N, T, H):
    log(f"block norm N={N} T={T} H={H}")
    sh, x, res, gp, gate, gn, dy, dr = norm_case(N, T, H, T)
    r_out, y = check_norm(sh, x, res, gp, None, -1.25, gn)
    got = check_norm_grad(sh, dy, dr, x, res, gp, None, -1.25, gn)
    a, b = x.clone(), res.clone()
    moe.moe_block_norm(sh, a, b, gp, None, -1.25, gn, 1e-5, b, a)
    assert torch.equal(b, r_out) and torch.equal(a, y)
    ws = torch.empty(moe.moe_block_norm_grad_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    dg = [torch.empty(H, device="cuda") for _ in range(2)]
    moe.moe_block_norm_grad(sh, dy, dr, x, res, gp, None, -1.25, gn, 1e-5, dy, dr, None, *dg, ws)
    assert torch.equal(dy, got["dx"]) and torch.equal(dr, got["dresidual"])
    assert torch.equal(dg[0], got["dgamma_post"]) and torch.equal(dg[1], got["dgamma_next"])


def test_block_norm_parts():
    """Without a next norm, without a gradient from behind, alpha of 0."""
    log("block norm parts")
    sh, x, res, gp, gate, gn, dy, dr = norm_case(2, 40, 640, 1)
    r1, _ = check_norm(sh, x, res, gp, gate, 1.0, None)
    r2, _ = check_norm(sh, x, res, gp, gate, 1.0, gn)
    assert torch.equal(r1, r2)
    check_norm_grad(sh, None, dr, x, res, gp, gate, 1.0, None)
    check_norm_grad(sh, dy, None, x, res, gp, gate, 1.0, gn)
    check_norm(sh, x, res, gp, gate, 0.0, gn)
    assert (check_norm_grad(sh, dy, dr, x, res, gp, gate, 0.0, gn)["dresidual"] == 0).all()
    check_norm_grad(sh, dy, dr, x, res, gp, torch.zeros_like(gate), 1.0, gn)


def test_block_norm_grad_where_the_terms_cancel():
    """residual = -gate * (x / rms(x) * gamma_post) but for a bf16 rounding and a
    few columns: r is small beside both of its terms."""
    log("block norm cancelling")
    N, T, H = 2, 9, 1024
    sh, x, res, gp, gate, gn, dy, dr = norm_case(N, T, H, 3)
    x = normal((N, T, H), gen(4))
    n1 = x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-5) * gp.double()
    res = (-gate.double()[..., None] * n1).to(BF)
    res[..., :8] = 0
    check_norm(sh, x, res, gp, gate, 1.0, gn)
    check_norm_grad(sh, dy, dr, x, res, gp, gate, 1.0, gn)


def test_block_norm_values():
    """Rows of zeros, infinities and NaN, each on its own."""
    H = 512
    sh, x, res, gp, gate, gn, dy, dr = norm_case(1, 5, H, 2)
    x[0, 0], res[0, 0] = 0, 0
    x[0, 1, 3] = float("inf")
    res[0, 2, 7] = float("nan")
    r, y = torch.empty_like(x), torch.empty_like(x)
    moe.moe_block_norm(sh, x, res, gp, gate, 0.5, gn, 1e-6, r, y)
    assert (r[0, 0] == 0).all() and (y[0, 0] == 0).all()
    assert r[0, 1, 3].isnan() and y[0, 1].isnan().all() and y[0, 2].isnan().all()
    ok = slice(3, 5)
    rv, br, yv, by = R.block_norm(x[:, ok], res[:, ok], gp, gate[:, ok], 0.5, gn, 1e-6)
    X.check_bf16(r[:, ok], rv, br, "r")
    X.check_bf16(y[:, ok], yv, by, "y")
    out = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(gate)] + [torch.empty(H, device="cuda") for _ in range(2)]
    ws = torch.empty(moe.moe_block_norm_grad_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    moe.moe_block_norm_grad(sh, dy, dr, x, res, gp, gate, 0.5, gn, 1e-6, *out, ws)
    want = R.block_norm_grad(dy[:, ok], dr[:, ok], x[:, ok], res[:, ok], gp, gate[:, ok], 0.5, gn, 1e-6)
    X.check_bf16(out[0][:, ok], *want["dx"], "dx")
    X.check_bf16(out[1][:, ok], *want["dresidual"], "dresidual")
    assert out[0][0, 0].isfinite().all() and out[3].isnan().all()


def test_no_tokens():
    sh = moe.shape(2, 0, 256, 4, 2)
    dw = torch.ones((4, 64, 128), dtype=BF, device="cuda")
    moe.moe_grouped_wgrad(sh, None, None, None, 64, 128, dw, add=True)
    assert (dw == 1).all()
    moe.moe_grouped_wgrad(sh, None, None, None, 64, 128, dw)
    assert (dw == 0).all()
    g = torch.ones(256, dtype=BF, device="cuda")
    out = [torch.ones(256, device="cuda") for _ in range(2)]
    ws = torch.empty(moe.moe_block_norm_grad_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    moe.moe_block_norm_grad(sh, None, None, None, None, g, None, 1.0, g, 1e-6, None, None, None, *out, ws)
    assert (out[0] == 0).all() and (out[1] == 0).all()


# ------------------------------------------------------------------ together

class Layer:
    """One layer's step as a user's program runs it, on the library's calls."""

    def __init__(self, N, T, E, k, H, I, seed):  # noqa: E741
        self.dims = N, T, E, k, H, I
        self.sh, self.B, self.idx, self.w = routed(N, T, E, k, H, seed)
        g = gen(seed)
        rows = moe.moe_recv_rows(self.sh)
        self.tokens, self.residual = normal((N, T, H), g), normal((N, T, H), g, 2.0)
        self.w13, self.w2 = normal((E, 2 * I, H), g, H ** -0.5), normal((E, H, I), g, I ** -0.5)
        self.gp, self.gn = ((1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF) for _ in range(2))
        self.gate = torch.sigmoid(torch.randn((N, T), generator=g, device="cuda"))
        self.dy, self.dres = normal((N, T, H), g), normal((N, T, H), g)
        e = lambda *s, t=BF: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        f = torch.float32
        self.x, self.a, self.y, self.y_em, self.dy_em = e(rows, H), e(rows, I), e(N, T, H), e(rows, H), e(rows, H)
        self.h_q, self.h_s = e(rows, 2 * I, t=torch.uint8), e(rows, 2 * I // 128, t=f)
        self.out, self.r = e(N, T, H), e(N, T, H)
        self.dh, self.dx = e(rows, 2 * I), e(rows, H)
        self.ones = torch.ones((N, T, k), device="cuda")
        self.ws = e(moe.moe_block_norm_grad_workspace_bytes(self.sh), t=torch.uint8)
        self.g = {"tokens": e(N, T, H), "residual": e(N, T, H), "w13": e(E, 2 * I, H, t=f), "w2": e(E, H, I, t=f),
                  "w": e(N, T, k, t=f), "gate": e(N, T, t=f), "gp": e(H, t=f), "gn": e(H, t=f)}
        self.dout = e(N, T, H)

    def step(self):
        N, T, E, k, H, I = self.dims  # noqa: E741
        sh, B, g = self.sh, self.B, self.g
        moe.moe_dispatch_direct(sh, None, self.idx, None, None, B.send_pos, B.exp_off, B.row_src, B.ws)
        route = (self.idx, B.send_pos)
        moe.moe_combine_grad(sh, self.tokens, None, *route, None, B.row_src, B.ws, self.x, None)
        moe.moe_ffn_up(sh, self.x, self.w13, B.exp_off, H, I, self.a, self.h_q, self.h_s)
        moe.moe_grouped_gemm_bf16(sh, self.a, self.w2, B.exp_off, I, H, False, self.y_em)
        moe.moe_combine_pull(sh, self.y_em, *route, self.w, B.ws, self.out)
        moe.moe_block_norm(sh, self.out, self.residual, self.gp, self.gate, 0.75, self.gn, 1e-6, self.r, self.y)
        moe.moe_block_norm_grad(sh, self.dy, self.dres, self.out, self.residual, self.gp, self.gate, 0.75, self.gn,
                                1e-6, self.dout, g["residual"], g["gate"], g["gp"], g["gn"], self.ws)
        moe.moe_combine_grad(sh, self.dout, self.y_em, *route, self.w, B.row_src, B.ws, self.dy_em, g["w"])
        moe.moe_ffn_up_grad(sh, self.dy_em, self.w2, self.h_q, self.h_s, B.exp_off, H, I, self.dh, self.a)
        moe.moe_grouped_gemm_bf16(sh, self.dh, self.w13, B.exp_off, 2 * I, H, True, self.dx)
        moe.moe_grouped_wgrad(sh, self.dh, self.x, B.exp_off, 2 * I, H, g["w13"])
        moe.moe_grouped_wgrad(sh, self.dy_em, self.a, B.exp_off, H, I, g["w2"])
        moe.moe_combine_pull(sh, self.dx, *route, self.ones, B.ws, g["tokens"])

    def results(self):
        return {"r": self.r, "y": self.y, **self.g}

    def exact(self):
        """The same step by automatic differentiation in 64 bits."""
        N, T, E, k, H, I = self.dims  # noqa: E741
        v = {n: getattr(self, n).double().requires_grad_() for n in self.g}
        tok, idx = v["tokens"].view(-1, H), self.idx.view(-1, k).long()
        out = torch.zeros_like(tok)
        for e in range(E):
            t, j = (idx == e).nonzero(as_tuple=True)
            h = tok[t] @ v["w13"][e].T
            y = (h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]) @ v["w2"][e].T
            out = out.index_add(0, t, y * v["w"].view(-1, k)[t, j, None])
        out = out.view(N, T, H)
        r, _, y, _ = R.block_norm(out, v["residual"], v["gp"], v["gate"], 0.75, v["gn"], 1e-6)
        ((y * self.dy.double()).sum() + (r * self.dres.double()).sum()).backward()
        return {"r": r.detach(), "y": y.detach(), **{n: t.grad for n, t in v.items()}}


@pytest.mark.parametrize("N,T,E,k,H,I", [(2, 70, 8, 2, 512, 256), (4, 300, 8, 4, 256, 384)])
def test_layer_forwards_and_backwards(N, T, E, k, H, I):  # noqa: E741
    log(f"layer N={N} T={T} E={E} k={k} H={H} I={I}")
    L = Layer(N, T, E, k, H, I, T)
    L.step()
    got, want = L.results(), L.exact()
    # r and y pass four bf16 roundings at most (a, y_em, out, themselves).
    for n in ("r", "y"):
        R.near(got[n], want[n], 4, n)
    # Gradients behind the checkpoint take its 8-bit values: half a step of e4m3
    # is 2^-4 of a value, spread evenly 2^-4 / sqrt(3) of the norm; silu's slope
    # and its change (|silu''| <= 1/2) carry that to dh at most twice (g and u).
    for n, t in got.items():
        rel = ((t.double() - want[n]).norm() / want[n].norm()).item()
        log(f"  {n}: {rel:.2e} of the norm")
        if n in ("residual", "gate", "gp", "gn"):
            R.near(t, want[n], 8, n)
        elif n == "w":
            R.near(t, want[n], 8, n)
        elif n in ("tokens", "w13", "w2"):
            assert rel <= 2 * X.E4M3_HALF / 3 ** 0.5, n


def test_layer_replayed_and_on_another_stream():
    """A captured step replayed several times, with eager work between, and a
    step on a side stream, give the eager step's bytes."""
    L = Layer(2, 64, 8, 2, 256, 128, 4)
    L.step()
    torch.cuda.synchronize()
    ref = {n: t.clone() for n, t in L.results().items()}
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        L.step()
    s.synchronize()
    assert all(torch.equal(t, ref[n]) for n, t in L.results().items())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step()
    for i in range(4):
        for t in L.results().values():
            t.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, ref[n]) for n, t in L.results().items()), i
        L.step()
        torch.cuda.synchronize()
        assert all(torch.equal(t, ref[n]) for n, t in L.results().items()), i
