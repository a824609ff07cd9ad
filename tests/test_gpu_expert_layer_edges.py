"""The expert layer's operators on the GPU at the ends of the number range, on
the tile and pass variants that few shapes reach, and under loads that gather
on a few experts; against the float64 forms of tests/expert_ref.py."""
import pytest
import torch

import combine_lds_atomic_amd as moe
import expert_ref as X

pytestmark = pytest.mark.gpu

from gpu_harness import log  # noqa: E402
from test_gpu_expert_layer import (CHAIN, check_layer, layer_inputs, make_groups, run_chain, run_gemm,  # noqa: E402
                                   run_layer, uneven)

TINY = 2.0 ** -149       # float32's smallest step


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def check_tiny_rows(q, s, v, dv):
    """8-bit rows whose scales are near or below float32's smallest normal
    number.  The scale amax / 448 is off by half of float32's smallest step
    besides the value's own error, and 448 times that by at most
    448 * 2^-150, which is also how far the saturated bytes of a block may
    stay behind its largest values."""
    b, db = v.reshape(v.shape[0], -1, 128), dv.reshape(v.shape[0], -1, 128)
    amax, near = b.abs().amax(-1), db.amax(-1)
    s = s.double()
    off = (s - amax / 448.0).abs()
    assert bool((off <= near / 448.0 + TINY / 2 + 4 * X.U * amax / 448.0).all()), f"scale off by {off.max().item()}"
    assert not bool(((q & 0x7F) == 0x7F).any()), f"{int(((q & 0x7F) == 0x7F).sum())} bytes are NaN"
    got = q.view(X.F8).double().reshape(b.shape) * s[..., None]
    lim = X.E4M3_HALF * (b.abs() + db) + X.E4M3_SUB * 1.01 * s[..., None] + 448.0 * TINY / 2 + 3 * db
    d = (got - b).abs()
    assert bool((d <= lim).all()), f"{int((d > lim).sum())} bytes off, worst {(d / lim).max().item()}"


@pytest.fixture(autouse=True)
def no_nan_bytes(monkeypatch):
    """A NaN byte beside a finite scale passes a comparison that asks whether
    the difference is above a limit; here every 8-bit row is also looked at
    for such bytes."""
    check = X.check_quantised

    def strict(q, s, v, dv, what=""):
        nan = ((q & 0x7F) == 0x7F).reshape(*s.shape, 128) & s.isfinite()[..., None]
        assert not bool(nan.any()), f"{what}: {int(nan.sum())} bytes are NaN"
        check(q, s, v, dv, what)
    monkeypatch.setattr(X, "check_quantised", strict)


# ------------------------------------------------------------------ subnormal scales

def test_norm_subnormal_scales():
    """Block maxima from about 1e-43 to 1e-39: the scales have one to a dozen
    bits, and quotients reach 1.5 times 448."""
    R, H = 48, 1280
    log(f"norm R={R} H={H}, subnormal scales")
    g = gen(91)
    down = torch.arange(10, device="cuda")[None, :, None] * 1.4         # the first block sets the row's norm
    x = (torch.randn((R, 10, 128), generator=g, device="cuda") * 2.0 ** -down).reshape(1, R, H).bfloat16()
    gamma = torch.full((H,), 3 * 2.0 ** -133, device="cuda").bfloat16()
    assert (gamma.double() == 3 * 2.0 ** -133).all()
    sh = moe.shape(1, R, H, 1, 1)
    q = torch.empty((1, R, H), dtype=torch.uint8, device="cuda")
    s = torch.empty((1, R, H // 128), device="cuda")
    moe.moe_rmsnorm_quant(sh, x, None, gamma, 1e-6, None, None, q, s)
    _, n, rel = X.norm(x[0], None, gamma, 1e-6)
    amax = n.abs().reshape(R, -1, 128).amax(-1)
    assert float(amax.min()) < 8e-43 and float(amax.max()) > 1e-40      # the range the test is about
    check_tiny_rows(q[0], s[0], n, n.abs() * rel + TINY)


@pytest.mark.parametrize("E,T,I", [(1, 24, 256), (1, 200, 256), (64, 32768, 512)])   # narrow, middle and large tile
def test_swiglu_subnormal_scales(E, T, I):  # noqa: E741
    """The activation is quadratic in a small input's scale: block maxima from
    3e-43 to 2e-41."""
    log(f"swiglu E={E} T={T} I={I}, subnormal scales")
    g = gen(92 + T)
    K, n = 256, T // E
    sh = moe.shape(1, T, 128, E, 1)
    eo = (torch.arange(E + 1, device="cuda") * n).int()[None]
    groups = [(e, e * n, n) for e in range(E)]
    x_q, _ = X.quantise(torch.randn((T, K), generator=g, device="cuda"))
    w_q, w_s = X.weights(E, 2 * I, K, g)
    one = torch.ones((T, K // 128), device="cuda")
    most = torch.empty(T, dtype=torch.float64, device="cuda")
    for sl, h, _ in X.gemm(x_q, one, w_q, w_s, groups):
        most[sl] = (h[:, :I] * h[:, I:]).abs().amax(1) / 2
    want = torch.logspace(-42.5, -40.7, T, device="cuda", dtype=torch.float64)
    x_s = (want / most).sqrt().float()[:, None].expand(T, K // 128).contiguous()
    q, s = torch.empty((T, I), dtype=torch.uint8, device="cuda"), torch.empty((T, I // 128), device="cuda")
    moe.moe_grouped_gemm_swiglu(sh, x_q, x_s, w_q, w_s, eo, K, I, q, s)
    for sl, a, da in X.swiglu(x_q, x_s, w_q, w_s, groups):
        check_tiny_rows(q[sl], s[sl], a, da + TINY)


# ------------------------------------------------------------------ one quantiser

def test_norm_rows_are_dispatchs_bytes():
    """A row of ones has norm 1, so y is gamma itself; the norm's 8-bit rows
    then hold the same values as dispatch's of y, and the same bytes."""
    H, T = 32768, 1
    log(f"norm against dispatch H={H}")
    g = gen(93)
    bits = [torch.randint(0, 1 << 16, (H,), generator=g, device="cuda")]                       # every exponent in a block
    bits.append(torch.randint(0x3C00, 0x4200, (H,), generator=g, device="cuda"))               # near 1
    bits[1] += torch.randint(0, 2, (H,), generator=g, device="cuda") << 15
    bits.append(torch.randint(0, 0x100, (H,), generator=g, device="cuda"))                     # subnormal, many zeros
    bits[2] *= torch.randint(0, 2, (H,), generator=g, device="cuda")
    bits.append(torch.randint(1, 5, (H,), generator=g, device="cuda"))                         # the smallest numbers
    bits.append((torch.randint(0, 2, (H,), generator=g, device="cuda") << 15) + torch.repeat_interleave(
        torch.randint(0, 0x7F80, (H // 128,), generator=g, device="cuda"), 128))               # one magnitude a block
    sh = moe.shape(1, T, H, 1, 1)
    x = torch.ones((1, T, H), dtype=torch.bfloat16, device="cuda")
    B = moe.allocate(sh, "cuda")
    idx = torch.zeros((1, T, 1), dtype=torch.int32, device="cuda")
    for b in bits:
        b = torch.where((b & 0x7F80) == 0x7F80, b & 0xBFFF, b)                                  # finite
        gamma = torch.where(b >= 1 << 15, b - (1 << 16), b).to(torch.int16).view(torch.bfloat16)
        y = torch.empty_like(x)
        q, s = torch.empty((1, T, H), dtype=torch.uint8, device="cuda"), torch.empty((1, T, H // 128), device="cuda")
        moe.moe_rmsnorm_quant(sh, x, None, gamma, 1e-12, None, y, q, s)
        assert torch.equal(y.view(torch.int16).flatten(), gamma.view(torch.int16))
        moe.moe_dispatch_direct(sh, y, idx, B.x_q, B.x_s, B.send_pos, B.exp_off, B.row_src, B.ws)
        assert torch.equal(B.x_q.flatten()[:H].view(torch.uint8), q.flatten())
        assert torch.equal(B.x_s.flatten()[:H // 128], s.flatten())


# ------------------------------------------------------------------ sums of the plain product

@pytest.mark.parametrize("E,T,F", [(1, 9, 144), (1, 130, 144), (8, 16384, 4096)])   # narrow, middle and large tile
def test_product_with_outliers_that_cancel(E, T, F):
    """Two columns whose products are 448 * 448 and its negative, in different
    groups of eight columns: what the e4m3 matrix instruction drops of their
    neighbours is within the stated bound, and the other groups' products
    arrive as if there were no outlier."""
    log(f"product with outliers E={E} T={T} F={F}")
    g = gen(95 + T)
    K, n = 512, T // E
    f8 = lambda *s: (torch.randn(s, generator=g, device="cuda") * 0.5).to(X.F8).view(torch.uint8)  # noqa: E731
    x_q, w_q = f8(T, K), f8(E, F, K)
    x_s = torch.ones((T, K // 128), device="cuda")
    w_s = torch.ones((E, -(-F // 128), K // 128), device="cuda")
    plus, minus = 131, 203                        # columns of the second block, of its first and tenth group
    x_q[:, [plus, minus]] = 0x7E                  # 448
    w_q[:, :, plus], w_q[:, :, minus] = 0x7E, 0xFE
    eo = (torch.arange(E + 1, device="cuda") * n).int()[None]
    y = torch.empty((T, F), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm(moe.shape(1, T, 128, E, 1), x_q, x_s, w_q, w_s, eo, K, F, y)
    for e in range(E):
        rows, feats = slice(e * n, e * n + min(n, 130)), slice(F - 144, F)
        xv, wv = X.values(x_q[rows], x_s[rows]), X.values(w_q[e], w_s[e], 128)[feats]
        # the outliers' own sum is exact in float32, so the sums round what is left: the groups' sums on
        # 2^-23 of the 2^18 that passes through, then the blocks
        ref = xv @ wv.T
        d = X.e4m3_loss(xv, wv) + 16 * 2.0 ** (18 - 23)
        lim = X.BF16_HALF * (ref.abs() + d) + d
        off = (y[rows, feats].double() - ref).abs()
        assert bool((off <= lim).all()), f"expert {e}: worst {(off / lim).max().item()}"


# ------------------------------------------------------------------ tile variants

@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N,E,T,k,K,F", [
    (4, 384, 4096, 4, 384, 256),        # more than 256 experts, 170 rows on average, uneven: the middle tile
    (2, 300, 375, 20, 1152, 128),       # 50 on average, an expert count that no lane count divides
    (1, 257, 100, 64, 256, 384),        # 24 on average: the plain form's middle, SwiGLU's narrow tile
    (1, 260, 195, 64, 256, 128),        # 48 on average: SwiGLU's narrow tile at its upper end
    (2, 100, 100, 6, 512, 384),         # 12 on average: the plain form's narrow tile at its upper end
])
def test_products_of_many_uneven_experts(swiglu, N, E, T, k, K, F):
    log(f"gemm swiglu={swiglu} N={N} E={E} T={T} k={k} K={K} F={F}")
    counts = uneven(E, N * T * k, T, zero_every=5)
    assert max(counts) > 3 * N * T * k // E and min(counts) == 0
    run_gemm(N, E, counts, K, F, T, k, swiglu=swiglu, seed=E)


@pytest.mark.parametrize("N,E,T,k,K,F", [(1, 1, 1, 1, 128, 128), (2, 8, 9, 2, 384, 256), (4, 16, 100, 4, 1024, 384),
                                         (2, 8, 2000, 2, 384, 4096), (4, 512, 19200, 2, 128, 256)])
def test_swiglu_bytes_are_numbers(N, E, T, k, K, F):
    """Each tile variant once more, with the look for NaN bytes."""
    log(f"swiglu bytes N={N} E={E} T={T} k={k} K={K} F={F}")
    run_gemm(N, E, uneven(E, N * T * k, T), K, F, T, k, swiglu=True, seed=K + 1)


# ------------------------------------------------------------------ infinities

def test_product_past_the_largest_numbers():
    """Sums beyond bf16's and float32's range become infinities of their sign,
    others of the row stay what they are, and so do the other rows."""
    g = gen(96)
    K, F, T = 128, 256, 5
    log("product past the largest numbers")
    x_q, x_s = X.quantise(torch.randn((T, K), generator=g, device="cuda"))
    w_q, w_s = X.weights(1, F, K, g)
    x_s[2] *= 2.5e38
    x_s[3] = float("inf")
    eo = make_groups(1, 1, [T])
    y = torch.empty((T, F), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm(moe.shape(1, T, 128, 1, 1), x_q, x_s, w_q, w_s, eo, K, F, y)
    for sl, r, d in X.gemm(x_q, x_s, w_q, w_s, [(0, 0, 2), (0, 4, 1)]):
        assert bool(((y[sl].double() - r).abs() <= X.BF16_HALF * (r.abs() + d) + d).all())
    xv, wv = X.values(x_q[2:3], x_s[2:3]), X.values(w_q[0], w_s[0], 128)
    r = (xv @ wv.T)[0]
    d = X.e4m3_loss(xv, wv)[0] + r.abs() * 4 * X.U
    top = float(torch.finfo(torch.bfloat16).max) * (1 + 2.0 ** -9)      # from here on bf16 rounds to infinity
    over, under = r.abs() - d > top, r.abs() + d < top
    assert int(over.sum()) > 10 and int(under.sum()) > 100 and int((~(over | under)).sum()) < 10
    got = y[2].double()
    assert bool((got[over] == torch.sign(r[over]) * float("inf")).all())
    assert bool(((got - r).abs() <= X.BF16_HALF * (r.abs() + d) + d)[under].all())
    assert not bool(y[3].isfinite().any())


@pytest.mark.parametrize("T", [5, 40])
def test_swiglu_past_the_largest_numbers(T):
    """An activation beyond float32's range makes its block's scale infinite and
    its byte NaN; an infinite gate or up makes the block infinite or NaN; the
    other rows are what they were."""
    g = gen(97)
    K, I = 128, 256  # noqa: E741
    log(f"swiglu past the largest numbers T={T}")
    sh, eo = moe.shape(1, T, 128, 1, 1), make_groups(1, 1, [T])
    x_q, x_s = X.quantise(torch.randn((T, K), generator=g, device="cuda"))
    w_q, w_s = X.weights(1, 2 * I, K, g)

    def go(x_s, w_s):
        q, s = torch.empty((T, I), dtype=torch.uint8, device="cuda"), torch.empty((T, I // 128), device="cuda")
        moe.moe_grouped_gemm_swiglu(sh, x_q, x_s, w_q, w_s, eo, K, I, q, s)
        return q, s
    q0, s0 = go(x_s, w_s)
    big = x_s.clone()
    big[2] *= 1e30                       # gate and up about 1e30, their product 1e60 where the gate is positive
    big[3] = float("inf")                # every gate and up infinite
    q, s = go(big, w_s)
    keep = [t for t in range(T) if t not in (2, 3)]
    assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep])
    h = (X.values(x_q[2:3], big[2:3]) @ X.values(w_q[0], w_s[0], 128).T)[0]
    gate, up = h[:I], h[I:]
    assert float(gate.abs().min()) > 1e26 and float(up.abs().min()) > 1e26      # none is near zero
    assert bool((s[2] == float("inf")).all())
    assert bool((((q[2] & 0x7F) == 0x7F) == (gate > 0)).all()) and bool(((q[2] & 0x7F)[gate < 0] == 0).all())
    assert not bool(s[3].isfinite().any())
    for half in (0, 1):                  # an infinite scale of one block of gate, or of up, weights
        bad = w_s.clone()
        bad[0, half * (I // 128)] = float("inf")
        q, s = go(x_s, bad)
        assert not bool(s[:, 0].isfinite().any())
        assert torch.equal(q[:, 128:], q0[:, 128:]) and torch.equal(s[:, 1:], s0[:, 1:])


# ------------------------------------------------------------------ few-token layer under uneven loads

def check_load(N, T, H, E, k, I, gather, seed):  # noqa: E741
    """`gather`: (tokens, experts) that the first so many tokens choose alike."""
    log(f"layer N={N} T={T} H={H} E={E} k={k} I={I} gather={gather}")
    a = list(layer_inputs(N, T, H, E, k, I, seed=seed))
    if gather:
        n, chosen = gather
        a[1].view(-1, k)[:n, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32, device="cuda")
    out, flags = run_layer(N, T, H, E, k, I, *a)
    assert flags == 0
    check_layer(out, N, T, H, k, *a)
    again, _ = run_layer(N, T, H, E, k, I, *a)
    assert torch.equal(out, again)


@pytest.mark.parametrize("N,T,H,E,k,I,gather", [
    (1, 64, 1024, 32, 8, 2048, None),                        # 16 members: two column tiles, two weight tiles a workgroup
    (4, 16, 1152, 32, 8, 2048, (64, [5])),                   # ... one expert with all 64: a second pass over both
    (1, 64, 640, 32, 20, 2048, None),                        # 40 members: four column tiles, two weight tiles
    (1, 64, 384, 32, 24, 4096, (60, [31, 0, 7])),            # ... with four weight tiles, three experts nearly full
    (8, 8, 512, 256, 8, 2048, (64, [0, 9, 99, 100, 128, 200, 254, 255])),   # all on 8 of 256: four passes of one tile
    (1, 50, 256, 256, 4, 1024, (49, [17])),                  # 49 members of one tile: the last pass has one
    (2, 16, 128, 64, 2, 2048, (32, [63])),                   # one block of columns: three of four waves have none
])
def test_layer_uneven_loads(N, T, H, E, k, I, gather):  # noqa: E741
    check_load(N, T, H, E, k, I, gather, seed=H + E)


def test_layer_calls_on_two_streams_and_one_workspace_for_two_shapes():
    """Calls with workspaces of their own overlap freely; one workspace serves
    calls of several shapes in order, captured and replayed."""
    I = 384  # noqa: E741
    shapes = [(1, 9, 384, 24, 3, I), (1, 33, 256, 4, 2, I)]
    log(f"layer, two streams, shapes {shapes}")
    cases = []
    for i, c in enumerate(shapes):
        a = layer_inputs(*c, seed=50 + i)
        sh = moe.shape(*c[:5])
        cases.append((c, a, sh, torch.empty_like(a[0]), torch.empty(1, dtype=torch.int32, device="cuda")))
    want = [run_layer(*c, *a)[0] for c, a, *_ in cases]
    need = [moe.moe_layer_ll_workspace_bytes(sh, I) for _, _, sh, *_ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    own = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in need]
    torch.cuda.synchronize()
    for _ in range(5):
        for (_, a, sh, out, fl), ws, st in zip(cases, own, streams):
            moe.moe_layer_ll(sh, *a, I, out, fl, ws, stream=st)
    torch.cuda.synchronize()
    for (_, _, _, out, _), w in zip(cases, want):
        assert torch.equal(out, w)
        out.zero_()
    shared = torch.full((max(need),), 0xFF, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _, a, sh, out, fl in cases:
            moe.moe_layer_ll(sh, *a, I, out, fl, shared)
    for _ in range(3):
        shared.fill_(0xFF)
        for _, _, _, out, _ in cases:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for (_, _, _, out, _), w in zip(cases, want):
            assert torch.equal(out, w)


# ------------------------------------------------------------------ together, first and last step

@pytest.mark.parametrize("R", [0, 4 * 50 * 4])
def test_chain_norm_and_combine(R):
    """The first and last step of the layer that test_chain does not look at:
    the norm's outputs, and the combine of exactly the down product's rows."""
    log(f"chain R={R}: norm and combine")
    c = run_chain(CHAIN, 256, R)
    c["go"]()
    B, N, T, H, k = c["B"], CHAIN.N, CHAIN.T, CHAIN.H, CHAIN.k
    r, n, rel = X.norm(c["x"].view(-1, H), c["res"].view(-1, H), c["gamma"], 1e-6)
    X.check_bf16(c["res_out"].view(-1, H), r, r.abs() * X.U)
    X.check_bf16(c["y"].view(-1, H), n, n.abs() * rel)
    X.check_quantised(c["y_q"], c["y_s"], n, n.abs() * rel)
    comb = torch.zeros((N * T * k, H), dtype=torch.float64, device="cuda")
    src = B.row_src.long()
    comb[src[src >= 0]] = c["y_em"][src >= 0].double()
    at = B.send_pos.view(N, T * k).long() + torch.arange(N, device="cuda")[:, None] * (T * k)
    terms = comb[at.view(-1)].view(N * T, k, H) * c["w"].view(N * T, k, 1).double()
    ref = terms.sum(1)
    X.check_bf16(B.out.view(-1, H), ref, terms.abs().sum(1) * (2 * k * X.U))
