"""Host-side refusals of the expert layer's calls (no GPU needed: nothing is
launched): the C ABI's return codes, and the binding's checks of tensors."""
import ctypes

import pytest
import torch

import combine_lds_atomic_amd as moe

A = 0x10000000   # never dereferenced: every call below fails its host checks first
EINVAL, ENULL, EALIGN, ERANGE = -1, -2, -3, -4


def _p(v):
    return None if v is None else ctypes.c_void_p(v)


def _call(fn, sh, args):
    return getattr(moe.lib, fn)(ctypes.byref(sh), *[_p(a) if a is None or a >= A else a for a in args], None)


SH = moe.shape(2, 8, 256, 4, 2)
NORM = dict(x=A, residual=A, gamma=A, eps=1e-6, res_out=A, y=A, y_q=A, y_s=A)
GEMM = dict(x_q=A, x_s=A, w_q=A, w_s=A, exp_off=A, K=256, F=64, y=A)
SWIGLU = dict(x_q=A, x_s=A, w_q=A, w_s=A, exp_off=A, K=256, I=128, a_q=A, a_s=A)
LAYER = dict(tokens=A, idx=A, w=A, w13_q=A, w13_s=A, w2_q=A, w2_s=A, I=128, out=A, flags=A, ws=A)


def _norm(sh=SH, **kw):
    a = {**NORM, **kw}
    return moe.lib.moe_rmsnorm_quant(ctypes.byref(sh), _p(a["x"]), _p(a["residual"]), _p(a["gamma"]), a["eps"],
                                     _p(a["res_out"]), _p(a["y"]), _p(a["y_q"]), _p(a["y_s"]), None)


def test_norm_refusals():
    assert _norm(sh=moe.shape(2, 8, 200, 4, 2)) == EINVAL
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert _norm(eps=eps) == EINVAL
    assert _norm(x=None) == ENULL and _norm(gamma=None) == ENULL
    assert _norm(y_s=None) == ENULL and _norm(y_q=None) == ENULL        # one without the other
    assert _norm(y=None, y_q=None, y_s=None) == ENULL                   # nothing to write
    for n in ("x", "residual", "gamma", "res_out", "y", "y_q"):
        assert _norm(**{n: A + 8}) == EALIGN, n
    assert _norm(y_s=A + 2) == EALIGN
    assert _norm(sh=moe.shape(2, 0, 256, 4, 2), x=None, gamma=None) == 0


@pytest.mark.parametrize("fn,base", [("moe_grouped_gemm", GEMM), ("moe_grouped_gemm_swiglu", SWIGLU)])
def test_grouped_gemm_refusals(fn, base):
    def call(sh=SH, **kw):
        return _call(fn, sh, {**base, **kw}.values())
    out = "F" if "F" in base else "I"
    for K in (0, 64, 200, -128, 32768 + 128):
        assert call(K=K) == EINVAL, K
    for F in (0, 8, 40, -16, 32768 + 128):
        assert call(**{out: F}) == EINVAL, F
    if out == "I":
        assert call(I=192) == EINVAL      # half a scale block
    assert call(sh=moe.shape(3, 8, 256, 4, 2)) == EINVAL
    for n in base:
        if n not in ("K", "F", "I"):
            assert call(**{n: None}) == ENULL, n
            assert call(**{n: A + 2}) == EALIGN, n
    for n in ("x_q", "w_q", "y" if "y" in base else "a_q"):
        assert call(**{n: A + 8}) == EALIGN, n
    none = {n: None for n in base if n not in ("K", "F", "I")}
    assert call(sh=moe.shape(2, 0, 256, 4, 2), **none) == 0             # no rows: nothing to do
    assert call(sh=moe.shape(2, 0, 256, 4, 2), K=100, **none) == EINVAL


def test_layer_refusals():
    def call(sh=SH, **kw):
        return _call("moe_layer_ll", sh, {**LAYER, **kw}.values())
    for I in (0, 64, 200, -128, 32768 + 128):  # noqa: E741
        assert call(I=I) == EINVAL
        assert moe.lib.moe_layer_ll_workspace_bytes(ctypes.byref(SH), I) == EINVAL
    assert call(sh=moe.shape(5, 13, 256, 5, 2)) == EINVAL               # 65 tokens
    assert moe.lib.moe_layer_ll_workspace_bytes(ctypes.byref(moe.shape(1, 65, 256, 4, 2)), 128) == EINVAL
    assert moe.lib.moe_layer_ll_workspace_bytes(ctypes.byref(moe.shape(2, 1 << 30, 256, 4, 1)), 128) < 0
    for n in LAYER:
        if n != "I":
            assert call(**{n: None}) == ENULL, n
            assert call(**{n: A + 2}) == EALIGN, n
    for n in ("tokens", "w13_q", "w2_q", "out"):
        assert call(**{n: A + 8}) == EALIGN, n
    assert call(ws=A + 128) == EALIGN


def test_layer_workspace_holds_the_activation():
    for T, k, I in ((1, 8, 2048), (16, 2, 128), (64, 4, 640)):  # noqa: E741
        b = moe.moe_layer_ll_workspace_bytes(moe.shape(1, T, 256, 8, k), I)
        assert b >= 4 * T * k * I and b % 256 == 0


def test_binding_refuses_a_stream_of_another_device():
    """The kernels are launched for the current device; its streams only."""
    class Stream:
        cuda_stream = 0x1234

        def __init__(self, device_index):
            self.device_index = device_index
    assert moe._raw_stream(Stream(1), 1) == 0x1234
    with pytest.raises(ValueError, match="stream is on device 1, not on the current GPU"):
        moe._raw_stream(Stream(1), 0)


def test_binding_checks_tensors():
    """Type, contiguity, size and device are checked before a pointer is taken."""
    x = torch.zeros((2, 8, 256), dtype=torch.bfloat16)
    g = torch.zeros(256, dtype=torch.bfloat16)
    call = lambda x, g, y: moe.moe_rmsnorm_quant(SH, x, None, g, 1e-6, None, y, None, None)  # noqa: E731
    with pytest.raises(TypeError, match="x has type"):
        call(x.float(), g, x)
    with pytest.raises(TypeError, match="must be a tensor"):
        call(None, g, x)
    with pytest.raises(ValueError, match="x must be contiguous"):
        call(torch.zeros((2, 8, 512), dtype=torch.bfloat16)[..., ::2], g, x)
    with pytest.raises(ValueError, match="x has 2048 elements"):
        call(x[:1], g, x)
    with pytest.raises(ValueError, match="not on the current GPU"):
        call(x, g, x)
