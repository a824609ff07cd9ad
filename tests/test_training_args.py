"""Host-side refusals of the training calls (no GPU needed: nothing is
launched), and the 64-bit reference forms against automatic and numerical
differentiation."""
import ctypes

import pytest
import torch

import combine_lds_atomic_amd as moe
import expert_ref as X
import training_ref as R

A = 0x10000000   # never dereferenced: every call below fails its host checks first
EINVAL, ENULL, EALIGN, ERANGE = -1, -2, -3, -4
SH, EMPTY = moe.shape(2, 8, 256, 4, 2), moe.shape(2, 0, 256, 4, 2)

UP = dict(x=A, w13=A, exp_off=A, K=256, I=128, a=A, h_q=A, h_s=A)
GEMM = dict(x=A, w=A, exp_off=A, K=256, F=64, w_t=0, y=A)
UP_GRAD = dict(dy=A, w2=A, h_q=A, h_s=A, exp_off=A, K=256, I=128, dh=A, a=A)
WGRAD = dict(d=A, x=A, exp_off=A, F=64, K=48, dw=A, flags=0)
COMBINE = dict(dout=A, y_em=A, idx=A, send_pos=A, w=A, row_src=A, ws=A, dy_em=A, dw=A)
NORM = dict(x=A, residual=A, gamma_post=A, gate=A, alpha=0.5, gamma_next=A, eps=1e-6, res_out=A, y=A)
NORM_GRAD = dict(dy=A, dres=A, x=A, residual=A, gamma_post=A, gate=A, alpha=0.5, gamma_next=A, eps=1e-6, dx=A,
                 dresidual=A, dgate=A, dgamma_post=A, dgamma_next=A, ws=A)


def caller(fn, base):
    def call(sh=SH, **kw):
        a = {**base, **kw}.values()
        return getattr(moe.lib, fn)(ctypes.byref(sh), *[ctypes.c_void_p(v) if isinstance(v, int) and v >= A else v
                                                        for v in a], None)
    return call


def refused_alike(call, base, optional, by4, numbers, bad_shape=moe.shape(3, 8, 256, 4, 2)):
    """A bad shape, each array missing, each array badly aligned."""
    assert call(sh=bad_shape) == EINVAL
    for n in base:
        if n in numbers:
            continue
        if n not in optional:
            assert call(**{n: None}) == ENULL, n
        assert call(**{n: A + 2}) == EALIGN, n
        if n not in by4:
            assert call(**{n: A + 8}) == EALIGN, n


@pytest.mark.parametrize("fn,base,optional", [("moe_ffn_up", UP, ()), ("moe_ffn_up_grad", UP_GRAD, ("a",))])
def test_up_refusals(fn, base, optional):
    call = caller(fn, base)
    refused_alike(call, base, optional, ("exp_off", "h_s"), ("K", "I"))
    for n in ("K", "I"):
        for v in (0, 64, 200, -128, 32768 + 128):
            assert call(**{n: v}) == EINVAL, (n, v)
    none = {n: None for n in base if n not in ("K", "I")}
    assert call(sh=EMPTY, **none) == 0
    assert call(sh=EMPTY, **{**none, "K": 100}) == EINVAL


def test_gemm_refusals():
    call = caller("moe_grouped_gemm_bf16", GEMM)
    refused_alike(call, GEMM, (), ("exp_off",), ("K", "F", "w_t"))
    for K in (0, 64, 200, -128, 65536 + 128):
        assert call(K=K) == EINVAL, K
    for F in (0, 8, 40, -16, 32768 + 16):
        assert call(F=F) == EINVAL, F
    assert call(w_t=2) == EINVAL and call(w_t=-1) == EINVAL
    assert call(sh=EMPTY, x=None, w=None, exp_off=None, y=None) == 0


def test_wgrad_refusals():
    call = caller("moe_grouped_wgrad", WGRAD)
    refused_alike(call, WGRAD, (), ("exp_off",), ("K", "F", "flags"))
    for K in (0, 8, 40, -16, 32768 + 16):
        assert call(K=K) == EINVAL, K
    for F in (0, 8, 40, -16, 65536 + 16):
        assert call(F=F) == EINVAL, F
    for flags in (4, -1, 8):
        assert call(flags=flags) == EINVAL
    assert call(sh=EMPTY, d=None, x=None, exp_off=None, dw=None) == ENULL      # zeros are still to be written


def test_combine_grad_refusals():
    call = caller("moe_combine_grad", COMBINE)
    refused_alike(call, COMBINE, ("w", "row_src", "dy_em"), ("idx", "send_pos", "w", "row_src", "dw"), ())
    assert call(ws=A + 128) == EALIGN
    assert call(dy_em=None, y_em=None, dw=None) == ENULL                       # nothing to write
    assert call(sh=moe.shape(2, 8, 256, 4, 2, 20), row_src=None) == ENULL      # fixed regions need row_src
    assert call(sh=EMPTY, dout=None, y_em=None, idx=None, send_pos=None, w=None, dy_em=None, dw=None) == 0


def test_block_norm_refusals():
    call = caller("moe_block_norm", NORM)
    refused_alike(call, NORM, ("gate",), ("gate",), ("alpha", "eps"), moe.shape(2, 8, 200, 4, 2))
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == EINVAL
    for alpha in (float("nan"), float("-inf")):
        assert call(alpha=alpha) == EINVAL
    assert call(sh=EMPTY, x=None, residual=None, gamma_post=None, res_out=None) == 0


def test_block_norm_grad_refusals():
    call = caller("moe_block_norm_grad", NORM_GRAD)
    refused_alike(call, NORM_GRAD, ("gate", "dres", "dgate"), ("gate", "dgate", "dgamma_post", "dgamma_next"),
                  ("alpha", "eps"), moe.shape(2, 8, 200, 4, 2))
    assert call(eps=0.0) == EINVAL and call(alpha=float("inf")) == EINVAL
    assert call(ws=A + 128) == EALIGN
    assert call(dy=None, gamma_next=None, dgamma_next=None, dres=None) == ENULL    # no gradient at all
    assert call(dy=None) == ENULL                                                  # a next norm without its gradient
    big = moe.shape(16, 4096, 7168, 16, 1)
    assert moe.moe_block_norm_grad_workspace_bytes(big) >= 2 * 7168 * 4
    assert moe.lib.moe_block_norm_grad_workspace_bytes(ctypes.byref(moe.shape(2, 8, 200, 4, 2))) == EINVAL


def test_binding_checks_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    eo = torch.zeros((2, 3), dtype=torch.int32)
    up = lambda x, a: moe.moe_ffn_up(SH, x, bf(4, 256, 256), eo, 256, 128, a, None, None)  # noqa: E731
    with pytest.raises(TypeError, match="x has type"):
        up(bf(32, 256).float(), bf(32, 128))
    with pytest.raises(ValueError, match="x has 7936 elements, needs 8192"):
        up(bf(31, 256), bf(32, 128))
    with pytest.raises(ValueError, match="x must be contiguous"):
        up(bf(256, 32).T, bf(32, 128))
    with pytest.raises(ValueError, match="not on the current GPU"):
        up(bf(32, 256), bf(32, 128))
    with pytest.raises(TypeError, match="dw has type torch.float16"):
        moe.moe_grouped_wgrad(SH, bf(32, 64), bf(32, 48), eo, 64, 48, torch.zeros((4, 64, 48), dtype=torch.float16))
    with pytest.raises(TypeError, match="gate has type torch.float64"):
        moe._arg("moe_block_norm", "gate", torch.zeros(16).double(), (torch.float32,), 16, 0, True)


# ------------------------------------------------------------------ the reference's gradients

def _norm_inputs(rows=3, H=8):
    g = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(rows, H), r(rows, H), r(rows, H), r(rows, H), 1 + 0.3 * r(H), r(rows), 1 + 0.3 * r(H)


def test_block_norm_gradients_of_the_reference():
    dy, dr, x, res, gp, gate, gn = _norm_inputs()
    leaves = [v.clone().requires_grad_() for v in (x, res, gp, gate, gn)]
    r, _, y, _ = R.block_norm(leaves[0], leaves[1], leaves[2], leaves[3], 0.7, leaves[4], 1e-5)
    ((r * dr).sum() + (y * dy).sum()).backward()
    out = R.block_norm_grad(dy, dr, x, res, gp, gate, 0.7, gn, 1e-5)
    for n, leaf in zip(("dx", "dresidual", "dgamma_post", "dgate", "dgamma_next"), leaves):
        assert torch.allclose(out[n][0], leaf.grad, rtol=1e-10, atol=1e-12), n

    def loss(x):
        r, _, y, _ = R.block_norm(x, res, gp, gate, 0.7, gn, 1e-5)
        return (r * dr).sum() + (y * dy).sum()
    v = torch.randn(x.shape, generator=torch.Generator().manual_seed(8), dtype=torch.float64)
    slope = (loss(x + 1e-5 * v) - loss(x - 1e-5 * v)) / 2e-5
    assert torch.allclose(slope, (out["dx"][0] * v).sum(), rtol=1e-7)


def test_up_gradients_of_the_reference():
    g = torch.Generator().manual_seed(9)
    n, H, I = 5, 12, 128  # noqa: E741
    h_q, h_s = X.quantise(torch.randn((n, 2 * I), generator=g) * 2)
    w2, dy = torch.randn((H, I), generator=g, dtype=torch.float64), torch.randn((n, H), generator=g, dtype=torch.float64)
    dh, _, a, _ = R.up_grad(dy, w2, h_q, h_s)
    h = X.values(h_q, h_s).requires_grad_()
    act = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
    (act @ w2.T * dy).sum().backward()
    assert torch.allclose(a, act.detach(), rtol=1e-12) and torch.allclose(dh, h.grad, rtol=1e-9, atol=1e-12)
