"""The training operators where they went wrong once, or where a rarer form of a
kernel runs: against the plain float64 forms of tests/training_ref.py."""
import pytest
import torch

import combine_lds_atomic_amd as moe
import expert_ref as X
import test_gpu_training as base
import training_ref as R

pytestmark = pytest.mark.gpu

from gpu_harness import log  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("region_rows", [0, 1, 300])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_wgrad_no_tokens(region_rows, dtype):
    """An empty batch has no exp_off to read, with fixed regions either, and what
    the regions hold is nobody's: the weights' gradients are zeros, or what
    they were when added to."""
    log(f"wgrad without tokens, region_rows={region_rows} {dtype}")
    for N, E, F, K in ((1, 1, 16, 16), (2, 4, 64, 128), (4, 32, 272, 400)):
        sh = moe.shape(N, 0, 256, E, 1, region_rows)
        d, x = (torch.full((N * region_rows, n), float("nan"), dtype=BF, device="cuda") for n in (F, K))
        dw = torch.ones((E, F, K), dtype=dtype, device="cuda")
        moe.moe_grouped_wgrad(sh, d, x, None, F, K, dw, add=True)
        assert (dw == 1).all()
        moe.moe_grouped_wgrad(sh, d, x, None, F, K, dw)
        assert (dw == 0).all()


def test_wgrad_no_tokens_no_arrays():
    """The same with no arrays of rows at all."""
    sh = moe.shape(2, 0, 256, 4, 2, 50)
    dw = torch.ones((4, 64, 128), device="cuda")
    moe.moe_grouped_wgrad(sh, None, None, None, 64, 128, dw, add=True)
    assert (dw == 1).all()
    moe.moe_grouped_wgrad(sh, None, None, None, 64, 128, dw)
    assert (dw == 0).all()


def test_gates_whose_sigmoid_is_subnormal():
    """silu and its slope where 1 / (1 + exp(-g)) is below float32's normal range
    but exp(-g) is still in it: u of 1e30 brings the products back into bf16's."""
    log("subnormal sigmoids")
    H = I = 128  # noqa: E741
    parts = torch.tensor([[-80.0, 0.0], [-87.0, -0.25], [-87.0, -0.5], [-88.0, 0.0], [-88.5, 0.0], [-88.5, -0.1875]])
    n = len(parts)
    sh, eo = moe.shape(1, n, 128, 1, 1), torch.tensor([[0, n]], dtype=torch.int32, device="cuda")
    x = torch.zeros((n, H), dtype=BF, device="cuda")
    x[:, :2], x[:, 2] = parts.cuda().to(BF), 1.0
    w13, w2 = (torch.zeros(s, dtype=BF, device="cuda") for s in ((1, 2 * I, H), (1, H, I)))
    w13[0, :I, :2], w13[0, I:, 2], w2[0, 0] = 1.0, 1e30, 1.0
    dy = torch.zeros((n, H), dtype=BF, device="cuda")
    dy[:, 0] = 1.0
    a, dh, a2 = (torch.empty((n, m), dtype=BF, device="cuda") for m in (I, 2 * I, I))
    q, s = torch.empty((n, 2 * I), dtype=torch.uint8, device="cuda"), torch.empty((n, 2), device="cuda")
    moe.moe_ffn_up(sh, x, w13, eo, H, I, a, q, s)
    moe.moe_ffn_up_grad(sh, dy, w2, q, s, eo, H, I, dh, a2)

    def close(got, want, g):
        # the exponential's argument rounded twice (|g| 2^-23 of the result each way), some
        # twenty roundings, then bf16's half step; nothing cancels for g this far from 0
        lim = want.abs() * (X.BF16_HALF + (2 * g.abs() + 24) * R.U)
        bad = bool(((got.double() - want).abs() > lim).any())
        assert not bad, (got[:, 0].tolist(), want[:, 0].tolist())
    g = (x[:, :1].double() + x[:, 1:2].double()).expand(n, I)
    close(a, g * torch.sigmoid(g) * w13[0, I, 2].double(), g)
    h = X.values(q, s)
    g, u = h[:, :I], h[:, I:]
    t = torch.sigmoid(g)
    close(a2, g * t * u, g)
    close(dh[:, :I], u * t * (1 + g * (1 - t)), g)
    close(dh[:, I:], g * t, g)


# ------------------------------------------------------------------ norm gradients

@pytest.mark.parametrize("x_scale,g_scale,eps", [
    (1e15, 1e4, 1e-5),        # squares of x * gamma_post leave float32, those of x and of the outputs do not
    (1e10, 1e10, 1e-5),
    (1e-15, 1e-10, 1e-30),    # and those that vanish, with an eps that they count beside
])
@pytest.mark.parametrize("H", [1024, 8320, 20480])
def test_block_norm_grad_number_range(H, x_scale, g_scale, eps):
    log(f"block norm H={H} x of {x_scale} gamma of {g_scale}")
    g = base.gen(H)
    sh, N, T = moe.shape(1, 3, H, 1, 1), 1, 3
    x, res, dy, dr = (base.normal((N, T, H), g, s) for s in (x_scale, 4 * g_scale, 1.0, 1 / g_scale))
    gp, gn = (((1 + 0.2 * torch.randn(H, generator=g, device="cuda")) * s).to(BF) for s in (g_scale, 1.0))
    gate = torch.randn((N, T), generator=g, device="cuda")
    base.check_norm(sh, x, res, gp, gate, 0.75, gn, eps)
    base.check_norm_grad(sh, dy, dr, x, res, gp, gate, 0.75, gn, eps)


@pytest.mark.parametrize("N,T,H", [(2, 300, 8320), (1, 700, 16384), (1, 1300, 20480), (1, 600, 32768)])
def test_block_norm_many_wide_rows_and_in_place(N, T, H):
    """More than one row a workgroup, and outputs over inputs, in the forms that
    read a row again."""
    base.test_block_norm_many_rows_and_in_place(N, T, H)


@pytest.mark.parametrize("N,T,H", [(1, 300, 2048), (2, 300, 8320), (1, 9, 16384), (1, 300, 32768)])
def test_block_norm_grad_where_wide_rows_cancel(N, T, H):
    """Every second row's residual is minus the block's term but for a rounding and a
    few columns, so that both reductions alternate in a workgroup."""
    log(f"block norm cancelling N={N} T={T} H={H}")
    sh, x, res, gp, gate, gn, dy, dr = base.norm_case(N, T, H, H)
    x = base.normal((N, T, H), base.gen(4))
    n1 = x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-5) * gp.double()
    near = (-gate.double()[..., None] * n1).to(BF)
    near[..., :8] = 0
    res[:, ::2] = near[:, ::2]
    base.check_norm(sh, x, res, gp, gate, 1.0, gn)
    got = base.check_norm_grad(sh, dy, dr, x, res, gp, gate, 1.0, gn)
    ws = torch.empty(moe.moe_block_norm_grad_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    dgate, dgp, dgn = torch.empty_like(gate), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_block_norm_grad(sh, dy, dr, x, res, gp, gate, 1.0, gn, 1e-5, x, res, dgate, dgp, dgn, ws)
    for n, t in (("dx", x), ("dresidual", res), ("dgate", dgate), ("dgamma_post", dgp), ("dgamma_next", dgn)):
        assert torch.equal(t, got[n]), n


# ------------------------------------------------------------------ long sums

def chain_limit(K):
    """Relative to the norm of many sums of K products: an instruction takes 32
    products, in up to four groups that join the running sum one after the
    other.  Each join is off by half a float32 step at most, of a partial sum
    that is no larger in norm than the whole; independent, they add up as the
    root of their number.  Four more roundings for what follows the sum."""
    return R.U * ((4 * K / 32 / 3) ** 0.5 + 4)


@pytest.mark.parametrize("kind", ["any sign", "positive"])
def test_weight_gradients_of_many_rows(kind):
    """float32 gradients of an expert with tens of thousands of rows: the error
    grows as the root of the rows, not with their number."""
    log(f"wgrad of many rows, {kind}")
    g, counts, F, K = base.gen(8), [65536, 100, 30001], 272, 400
    rows = sum(counts)
    sh, eo = moe.shape(1, rows, 128, 3, 1), base.make_groups(1, 3, counts)
    d, x = base.normal((rows, F), g), base.normal((rows, K), g)
    if kind == "positive":
        d, x = d.abs(), x.abs()
    dw = torch.empty((3, F, K), device="cuda")
    moe.moe_grouped_wgrad(sh, d, x, eo, F, K, dw)
    for e, a, n in X.group_rows(eo, rows, 0):
        want = d[a:a + n].double().T @ x[a:a + n].double()
        rel = ((dw[e].double() - want).norm() / want.norm()).item()
        log(f"  {n} rows: {rel:.2e} of the norm")
        assert rel <= chain_limit(n)


@pytest.mark.parametrize("K", [7168, 32768])
def test_checkpoint_scales_of_the_large_tile(K):
    """h_s of the tile that has no registers to join its sums in parts."""
    log(f"checkpoint scales K={K}")
    g, rows, I = base.gen(K), 4096, 4096  # noqa: E741
    sh, eo = moe.shape(1, rows, 128, 1, 1), base.make_groups(1, 1, [rows])
    x, w13 = base.normal((rows, K), g), base.normal((1, 2 * I, K), g, K ** -0.5)
    a = torch.empty((rows, I), dtype=BF, device="cuda")
    q, s = torch.empty((rows, 2 * I), dtype=torch.uint8, device="cuda"), torch.empty((rows, 2 * I // 128), device="cuda")
    moe.moe_ffn_up(sh, x, w13, eo, K, I, a, q, s)
    some = torch.cat((torch.arange(100), torch.arange(rows - 100, rows))).cuda()
    h = x[some].double() @ w13[0].double().T
    want = h.view(len(some), -1, 128).abs().amax(-1) / 448
    rel = ((s[some].double() - want).norm() / want.norm()).item()
    log(f"  {rel:.2e} of the norm")
    assert rel <= chain_limit(K)
