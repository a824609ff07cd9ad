"""Python binding of libmoe_ep (MoE expert-parallel dispatch / combine on one
MI355X).  Argument marshalling only: every function forwards torch tensors'
device pointers and the current HIP stream to the C ABI of
``include/moe_ep.h`` under the same name; all computation happens in the HIP
kernels.  The expert layer's and the training functions also check each
tensor's type, contiguity, size and device, and the stream's device, first
(TypeError, ValueError).  Importing this module fails loudly if the library is not built.
"""
from __future__ import annotations

import ctypes
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_EP_LIB selects another build of the same library (e.g. a tuning variant).
LIB_PATH = os.environ.get("MOE_EP_LIB") or os.path.join(PKG, "libmoe_ep.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "moe_ep.h")

MOE_OK = 0
ERRORS = {-1: "MOE_EINVAL", -2: "MOE_ENULL", -3: "MOE_EALIGN", -4: "MOE_ERANGE", -5: "MOE_EHIP"}
WGRAD_F32, WGRAD_ADD = 1, 2
FLAG_BADID, FLAG_OVERFLOW, FLAG_BOUND, FLAG_TIMEOUT = 1, 2, 4, 8


class MoeError(RuntimeError):
    def __init__(self, fn: str, rc: int):
        super().__init__(f"{fn} returned {rc} ({ERRORS.get(rc, 'unknown')})")
        self.rc = rc


class moe_shape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("early_rows", ctypes.c_int32), ("region_rows", ctypes.c_int64)]

    def __repr__(self):
        return (f"moe_shape(N={self.N}, T={self.T}, H={self.H}, E={self.E}, k={self.k}, "
                f"region_rows={self.region_rows}, early_rows={self.early_rows})")


def shape(N: int, T: int, H: int, E: int, k: int, region_rows: int = 0, early_rows: int = 0) -> moe_shape:
    return moe_shape(N, T, H, E, k, early_rows, region_rows)


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python combine_lds_atomic_amd/build.py` "
                      "(or __graft_entry__.build()) first")

# torch ships its own HIP runtime.  It must be in the process before the
# library is opened, so that the library's libamdhip64.so.7 dependency binds to
# that same runtime (by soname) instead of loading a second one: with two
# runtimes the library sees no device and torch's streams mean nothing to it.
import torch  # noqa: E402,F401

lib = ctypes.CDLL(LIB_PATH)


def _hip_runtimes() -> set[str]:
    try:
        maps = open("/proc/self/maps").read()
    except OSError:  # pragma: no cover
        return set()
    return {ln.split()[-1] for ln in maps.splitlines() if "libamdhip64" in ln}


if len(_hip_runtimes()) > 1:
    raise ImportError(f"two HIP runtimes are loaded ({sorted(_hip_runtimes())}); import torch before anything "
                      "that links /opt/rocm's libamdhip64")

_P = ctypes.c_void_p
_S = ctypes.POINTER(moe_shape)
_SIG = {
    "moe_recv_rows": (ctypes.c_int64, [_S]),
    "moe_workspace_bytes": (ctypes.c_int64, [_S]),
    "moe_workspace_init": (ctypes.c_int, [_S, _P, _P]),
    "moe_dispatch_send": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P]),
    "moe_dispatch_send_ll": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P]),
    "moe_dispatch_direct": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_dispatch_direct_ll": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_dispatch_direct_noalloc": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_dispatch_recv": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_combine_send": (ctypes.c_int, [_S, _P, _P, _P, _P, _P]),
    "moe_combine_recv": (ctypes.c_int, [_S, _P, _P, _P, _P, _P]),
    "moe_combine_pull": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P]),
    "moe_combine_send_partial": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P]),
    "moe_combine_recv_partial": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P]),
    "moe_rmsnorm_quant": (ctypes.c_int, [_S, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P]),
    "moe_grouped_gemm": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, _P, _P]),
    "moe_grouped_gemm_swiglu": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, _P, _P, _P]),
    "moe_layer_ll_workspace_bytes": (ctypes.c_int64, [_S, ctypes.c_int32]),
    "moe_layer_ll": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _P]),
    "moe_ffn_up": (ctypes.c_int, [_S, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P]),
    "moe_grouped_gemm_bf16": (ctypes.c_int, [_S, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P]),
    "moe_ffn_up_grad": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, _P, _P, _P]),
    "moe_grouped_wgrad": (ctypes.c_int, [_S, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, _P, ctypes.c_int32, _P]),
    "moe_combine_grad": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_block_norm": (ctypes.c_int, [_S, _P, _P, _P, _P, ctypes.c_float, _P, ctypes.c_float, _P, _P, _P]),
    "moe_block_norm_grad_workspace_bytes": (ctypes.c_int64, [_S]),
    "moe_block_norm_grad": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, ctypes.c_float, _P, ctypes.c_float, _P, _P, _P,
                                           _P, _P, _P, _P]),
    "moe_status": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_uint32)]),
    "moe_layout_export": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P]),
}
for _name, (_res, _args) in _SIG.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def declared_symbols() -> list[str]:
    """Function names declared in include/moe_ep.h."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(moe_\w+)\s*\(", txt, re.M)))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _arg(fn, name, t, dtypes, count, dev, optional=False):
    """A tensor's device pointer, after the checks a raw pointer does not
    allow: type, contiguity, at least `count` elements, and memory of the
    current device `dev` (kernels run on the current device's streams)."""
    if t is None and (optional or count == 0):
        return None
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.is_contiguous() and t.numel() >= count \
            and t.get_device() == dev:
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{fn}: {name} must be a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{fn}: {name} has type {t.dtype}, wanted {' or '.join(str(d) for d in dtypes)}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous")
    if t.numel() < count:
        raise ValueError(f"{fn}: {name} has {t.numel()} elements, needs {count}")
    raise ValueError(f"{fn}: {name} is on {t.device}, not on the current GPU")


def _rows(sh) -> int:
    """Expert-major rows that a call reads or writes: an empty batch has none,
    whatever its fixed regions would hold (its arrays may be None)."""
    return moe_recv_rows(sh) if sh.T else 0


def _device() -> int:
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2   # -1 is the CPU's number


def _raw_stream(stream, dev):
    if stream is not None:
        if stream.device_index != dev:
            raise ValueError(f"stream is on device {stream.device_index}, not on the current GPU")
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else None


_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_F8 = (torch.uint8, torch.float8_e4m3fn)


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, rc: int) -> None:
    if rc != MOE_OK:
        raise MoeError(fn, rc)


# --------------------------------------------------------------- sizes

def moe_recv_rows(sh: moe_shape) -> int:
    r = lib.moe_recv_rows(ctypes.byref(sh))
    _check("moe_recv_rows", r if r < 0 else 0)
    return int(r)


def moe_workspace_bytes(sh: moe_shape) -> int:
    r = lib.moe_workspace_bytes(ctypes.byref(sh))
    _check("moe_workspace_bytes", r if r < 0 else 0)
    return int(r)


# --------------------------------------------------------------- entry points

def moe_workspace_init(sh, ws, stream=None):
    _check("moe_workspace_init", lib.moe_workspace_init(ctypes.byref(sh), _ptr(ws), _stream(stream)))


def moe_dispatch_send(sh, tokens, topk_idx, recv_q, recv_s, send_pos, ws, stream=None):
    _check("moe_dispatch_send", lib.moe_dispatch_send(ctypes.byref(sh), _ptr(tokens), _ptr(topk_idx), _ptr(recv_q),
                                                      _ptr(recv_s), _ptr(send_pos), _ptr(ws), _stream(stream)))


def moe_dispatch_send_ll(sh, tokens, topk_idx, recv_q, recv_s, send_pos, ws, stream=None):
    _check("moe_dispatch_send_ll", lib.moe_dispatch_send_ll(ctypes.byref(sh), _ptr(tokens), _ptr(topk_idx),
                                                            _ptr(recv_q), _ptr(recv_s), _ptr(send_pos), _ptr(ws),
                                                            _stream(stream)))


def moe_dispatch_direct(sh, tokens, topk_idx, x_q, x_s, send_pos, exp_off, row_src, ws, stream=None):
    _check("moe_dispatch_direct", lib.moe_dispatch_direct(ctypes.byref(sh), _ptr(tokens), _ptr(topk_idx), _ptr(x_q),
                                                          _ptr(x_s), _ptr(send_pos), _ptr(exp_off), _ptr(row_src),
                                                          _ptr(ws), _stream(stream)))


def moe_dispatch_direct_ll(sh, tokens, topk_idx, x_q, x_s, send_pos, exp_off, row_src, ws, stream=None):
    _check("moe_dispatch_direct_ll", lib.moe_dispatch_direct_ll(ctypes.byref(sh), _ptr(tokens), _ptr(topk_idx),
                                                                _ptr(x_q), _ptr(x_s), _ptr(send_pos), _ptr(exp_off),
                                                                _ptr(row_src), _ptr(ws), _stream(stream)))


def moe_dispatch_direct_noalloc(sh, tokens, topk_idx, x_q, x_s, send_pos, exp_off, row_src, flags, stream=None):
    _check("moe_dispatch_direct_noalloc", lib.moe_dispatch_direct_noalloc(
        ctypes.byref(sh), _ptr(tokens), _ptr(topk_idx), _ptr(x_q), _ptr(x_s), _ptr(send_pos), _ptr(exp_off),
        _ptr(row_src), _ptr(flags), _stream(stream)))


def moe_dispatch_recv(sh, recv_q, recv_s, ws, x_q, x_s, exp_off, row_src, stream=None):
    _check("moe_dispatch_recv", lib.moe_dispatch_recv(ctypes.byref(sh), _ptr(recv_q), _ptr(recv_s), _ptr(ws),
                                                      _ptr(x_q), _ptr(x_s), _ptr(exp_off), _ptr(row_src),
                                                      _stream(stream)))


def moe_combine_send(sh, y_em, row_src, ws, comb, stream=None):
    _check("moe_combine_send", lib.moe_combine_send(ctypes.byref(sh), _ptr(y_em), _ptr(row_src), _ptr(ws),
                                                    _ptr(comb), _stream(stream)))


def moe_combine_recv(sh, comb, send_pos, topk_w, out, stream=None):
    _check("moe_combine_recv", lib.moe_combine_recv(ctypes.byref(sh), _ptr(comb), _ptr(send_pos), _ptr(topk_w),
                                                    _ptr(out), _stream(stream)))


def moe_combine_pull(sh, y_em, topk_idx, send_pos, topk_w, ws, out, stream=None):
    _check("moe_combine_pull", lib.moe_combine_pull(ctypes.byref(sh), _ptr(y_em), _ptr(topk_idx), _ptr(send_pos),
                                                    _ptr(topk_w), _ptr(ws), _ptr(out), _stream(stream)))


def moe_combine_send_partial(sh, y_em, topk_idx, send_pos, topk_w, ws, comb, stream=None):
    _check("moe_combine_send_partial", lib.moe_combine_send_partial(ctypes.byref(sh), _ptr(y_em), _ptr(topk_idx),
                                                                    _ptr(send_pos), _ptr(topk_w), _ptr(ws),
                                                                    _ptr(comb), _stream(stream)))


def moe_combine_recv_partial(sh, comb, topk_idx, send_pos, ws, out, stream=None):
    _check("moe_combine_recv_partial", lib.moe_combine_recv_partial(ctypes.byref(sh), _ptr(comb), _ptr(topk_idx),
                                                                    _ptr(send_pos), _ptr(ws), _ptr(out),
                                                                    _stream(stream)))


def moe_rmsnorm_quant(sh, x, residual, gamma, eps, res_out, y, y_q, y_s, stream=None):
    f, dev = "moe_rmsnorm_quant", _device()
    n = sh.N * sh.T * sh.H
    _check(f, lib.moe_rmsnorm_quant(
        ctypes.byref(sh), _arg(f, "x", x, _BF16, n, dev), _arg(f, "residual", residual, _BF16, n, dev, True),
        _arg(f, "gamma", gamma, _BF16, sh.H if n else 0, dev), eps, _arg(f, "res_out", res_out, _BF16, n, dev, True),
        _arg(f, "y", y, _BF16, n, dev, True), _arg(f, "y_q", y_q, _F8, n, dev, True),
        _arg(f, "y_s", y_s, _F32, n // 128, dev, True), _raw_stream(stream, dev)))


def moe_grouped_gemm(sh, x_q, x_s, w_q, w_s, exp_off, K, F, y, stream=None):
    f, dev = "moe_grouped_gemm", _device()
    rows, kb = _rows(sh), K // 128
    E = sh.E if sh.T else 0
    _check(f, lib.moe_grouped_gemm(
        ctypes.byref(sh), _arg(f, "x_q", x_q, _F8, rows * K, dev), _arg(f, "x_s", x_s, _F32, rows * kb, dev),
        _arg(f, "w_q", w_q, _F8, E * F * K, dev), _arg(f, "w_s", w_s, _F32, E * -(-F // 128) * kb, dev),
        _arg(f, "exp_off", exp_off, _I32, sh.N + E if E else 0, dev), K, F, _arg(f, "y", y, _BF16, rows * F, dev),
        _raw_stream(stream, dev)))


def moe_grouped_gemm_swiglu(sh, x_q, x_s, w13_q, w13_s, exp_off, K, I, a_q, a_s, stream=None):  # noqa: E741
    f, dev = "moe_grouped_gemm_swiglu", _device()
    rows, kb, ib = _rows(sh), K // 128, I // 128
    E = sh.E if sh.T else 0
    _check(f, lib.moe_grouped_gemm_swiglu(
        ctypes.byref(sh), _arg(f, "x_q", x_q, _F8, rows * K, dev), _arg(f, "x_s", x_s, _F32, rows * kb, dev),
        _arg(f, "w13_q", w13_q, _F8, E * 2 * I * K, dev), _arg(f, "w13_s", w13_s, _F32, E * 2 * ib * kb, dev),
        _arg(f, "exp_off", exp_off, _I32, sh.N + E if E else 0, dev), K, I, _arg(f, "a_q", a_q, _F8, rows * I, dev),
        _arg(f, "a_s", a_s, _F32, rows * ib, dev), _raw_stream(stream, dev)))


def moe_layer_ll_workspace_bytes(sh: moe_shape, I: int) -> int:  # noqa: E741
    r = lib.moe_layer_ll_workspace_bytes(ctypes.byref(sh), I)
    _check("moe_layer_ll_workspace_bytes", r if r < 0 else 0)
    return int(r)


def moe_layer_ll(sh, tokens, topk_idx, topk_w, w13_q, w13_s, w2_q, w2_s, I, out, flags, ws, stream=None):  # noqa: E741
    f, dev = "moe_layer_ll", _device()
    n, H = sh.N * sh.T, sh.H
    need = moe_layer_ll_workspace_bytes(sh, I) if n else 0
    wq, wsc = (sh.E * I * H, sh.E * (I // 128) * (H // 128)) if n else (0, 0)
    _check(f, lib.moe_layer_ll(
        ctypes.byref(sh), _arg(f, "tokens", tokens, _BF16, n * H, dev),
        _arg(f, "topk_idx", topk_idx, _I32, n * sh.k, dev), _arg(f, "topk_w", topk_w, _F32, n * sh.k, dev),
        _arg(f, "w13_q", w13_q, _F8, 2 * wq, dev), _arg(f, "w13_s", w13_s, _F32, 2 * wsc, dev),
        _arg(f, "w2_q", w2_q, _F8, wq, dev), _arg(f, "w2_s", w2_s, _F32, wsc, dev), I,
        _arg(f, "out", out, _BF16, n * H, dev), _arg(f, "flags", flags, (torch.int32, torch.uint32), 1, dev),
        _arg(f, "ws", ws, (torch.uint8,), need, dev), _raw_stream(stream, dev)))


def moe_ffn_up(sh, x, w13, exp_off, K, I, a, h_q, h_s, stream=None):  # noqa: E741
    f, dev = "moe_ffn_up", _device()
    rows, E = _rows(sh), sh.E if sh.T else 0
    _check(f, lib.moe_ffn_up(
        ctypes.byref(sh), _arg(f, "x", x, _BF16, rows * K, dev), _arg(f, "w13", w13, _BF16, E * 2 * I * K, dev),
        _arg(f, "exp_off", exp_off, _I32, sh.N + E if E else 0, dev), K, I, _arg(f, "a", a, _BF16, rows * I, dev),
        _arg(f, "h_q", h_q, _F8, rows * 2 * I, dev, True), _arg(f, "h_s", h_s, _F32, rows * (2 * I // 128), dev, True),
        _raw_stream(stream, dev)))


def moe_grouped_gemm_bf16(sh, x, w, exp_off, K, F, w_t, y, stream=None):
    f, dev = "moe_grouped_gemm_bf16", _device()
    rows, E = _rows(sh), sh.E if sh.T else 0
    _check(f, lib.moe_grouped_gemm_bf16(
        ctypes.byref(sh), _arg(f, "x", x, _BF16, rows * K, dev), _arg(f, "w", w, _BF16, E * F * K, dev),
        _arg(f, "exp_off", exp_off, _I32, sh.N + E if E else 0, dev), K, F, bool(w_t),
        _arg(f, "y", y, _BF16, rows * F, dev), _raw_stream(stream, dev)))


def moe_ffn_up_grad(sh, dy, w2, h_q, h_s, exp_off, K, I, dh, a, stream=None):  # noqa: E741
    f, dev = "moe_ffn_up_grad", _device()
    rows, E = _rows(sh), sh.E if sh.T else 0
    _check(f, lib.moe_ffn_up_grad(
        ctypes.byref(sh), _arg(f, "dy", dy, _BF16, rows * K, dev), _arg(f, "w2", w2, _BF16, E * K * I, dev),
        _arg(f, "h_q", h_q, _F8, rows * 2 * I, dev), _arg(f, "h_s", h_s, _F32, rows * (2 * I // 128), dev),
        _arg(f, "exp_off", exp_off, _I32, sh.N + E if E else 0, dev), K, I,
        _arg(f, "dh", dh, _BF16, rows * 2 * I, dev), _arg(f, "a", a, _BF16, rows * I, dev, True),
        _raw_stream(stream, dev)))


def moe_grouped_wgrad(sh, d, x, exp_off, F, K, dw, add=False, stream=None):
    """dw's type, bfloat16 or float32, says which of the two is written."""
    f, dev = "moe_grouped_wgrad", _device()
    rows, E = _rows(sh), sh.E if sh.T else 0
    out = _arg(f, "dw", dw, _BF16 + _F32, sh.E * F * K, dev)
    _check(f, lib.moe_grouped_wgrad(
        ctypes.byref(sh), _arg(f, "d", d, _BF16, rows * F, dev), _arg(f, "x", x, _BF16, rows * K, dev),
        _arg(f, "exp_off", exp_off, _I32, sh.N + E if E else 0, dev), F, K, out,
        (WGRAD_F32 if dw is not None and dw.dtype == torch.float32 else 0) | (WGRAD_ADD if add else 0),
        _raw_stream(stream, dev)))


def moe_combine_grad(sh, dout, y_em, topk_idx, send_pos, topk_w, row_src, ws, dy_em, dtopk_w, stream=None):
    f, dev = "moe_combine_grad", _device()
    n, rows = sh.N * sh.T, _rows(sh)
    _check(f, lib.moe_combine_grad(
        ctypes.byref(sh), _arg(f, "dout", dout, _BF16, n * sh.H, dev),
        _arg(f, "y_em", y_em, _BF16, rows * sh.H, dev, True), _arg(f, "topk_idx", topk_idx, _I32, n * sh.k, dev),
        _arg(f, "send_pos", send_pos, _I32, n * sh.k, dev), _arg(f, "topk_w", topk_w, _F32, n * sh.k, dev, True),
        _arg(f, "row_src", row_src, _I32, rows, dev, True),
        _arg(f, "ws", ws, (torch.uint8,), moe_workspace_bytes(sh), dev),
        _arg(f, "dy_em", dy_em, _BF16, rows * sh.H, dev, True),
        _arg(f, "dtopk_w", dtopk_w, _F32, n * sh.k, dev, True), _raw_stream(stream, dev)))


def moe_block_norm(sh, x, residual, gamma_post, gate, alpha, gamma_next, eps, res_out, y, stream=None):
    f, dev = "moe_block_norm", _device()
    t = sh.N * sh.T
    n, H = t * sh.H, sh.H if t else 0
    _check(f, lib.moe_block_norm(
        ctypes.byref(sh), _arg(f, "x", x, _BF16, n, dev), _arg(f, "residual", residual, _BF16, n, dev),
        _arg(f, "gamma_post", gamma_post, _BF16, H, dev), _arg(f, "gate", gate, _F32, t, dev, True), alpha,
        _arg(f, "gamma_next", gamma_next, _BF16, H, dev, True), eps, _arg(f, "res_out", res_out, _BF16, n, dev),
        _arg(f, "y", y, _BF16, n, dev, True), _raw_stream(stream, dev)))


def moe_block_norm_grad_workspace_bytes(sh: moe_shape) -> int:
    r = lib.moe_block_norm_grad_workspace_bytes(ctypes.byref(sh))
    _check("moe_block_norm_grad_workspace_bytes", r if r < 0 else 0)
    return int(r)


def moe_block_norm_grad(sh, dy, dres_out, x, residual, gamma_post, gate, alpha, gamma_next, eps, dx, dresidual, dgate,
                        dgamma_post, dgamma_next, ws, stream=None):
    f, dev = "moe_block_norm_grad", _device()
    t, H = sh.N * sh.T, sh.H
    n = t * H
    _check(f, lib.moe_block_norm_grad(
        ctypes.byref(sh), _arg(f, "dy", dy, _BF16, n, dev, True), _arg(f, "dres_out", dres_out, _BF16, n, dev, True),
        _arg(f, "x", x, _BF16, n, dev), _arg(f, "residual", residual, _BF16, n, dev),
        _arg(f, "gamma_post", gamma_post, _BF16, H, dev), _arg(f, "gate", gate, _F32, t, dev, True), alpha,
        _arg(f, "gamma_next", gamma_next, _BF16, H, dev, True), eps, _arg(f, "dx", dx, _BF16, n, dev),
        _arg(f, "dresidual", dresidual, _BF16, n, dev), _arg(f, "dgate", dgate, _F32, t, dev, True),
        _arg(f, "dgamma_post", dgamma_post, _F32, H, dev),
        _arg(f, "dgamma_next", dgamma_next, _F32, H, dev, True),
        _arg(f, "ws", ws, (torch.uint8,), moe_block_norm_grad_workspace_bytes(sh), dev), _raw_stream(stream, dev)))


def moe_status(ws, stream=None) -> int:
    fl = ctypes.c_uint32(0)
    _check("moe_status", lib.moe_status(_ptr(ws), _stream(stream), ctypes.byref(fl)))
    return int(fl.value)


def moe_layout_export(sh, ws, cnt=None, send_off=None, recv_off=None, recv_total=None, base=None, stream=None):
    _check("moe_layout_export", lib.moe_layout_export(ctypes.byref(sh), _ptr(ws), _ptr(cnt), _ptr(send_off),
                                                      _ptr(recv_off), _ptr(recv_total), _ptr(base), _stream(stream)))


from .buffers import Buffers, allocate  # noqa: E402  (device-memory plumbing)
