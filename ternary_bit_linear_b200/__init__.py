"""Python binding of libtq -- the B200 (sm_100a) ternary linear layer.

Argument marshalling only: every function forwards torch CUDA tensors (their
device pointers) and the current CUDA stream to the C ABI declared in
include/tq.h and raises on a non-OK status.  All arithmetic runs in the CUDA
kernels of libtq.so.  There is no CPU fallback: if the library is missing or
the device is not sm_100, calls fail loudly.

The library is built in-tree by ``python -m ternary_bit_linear_b200.build``
(or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

GAMMA_PER_ROW = 1 << 0
FLAG_FWHT = 1 << 1
FLAG_RMSNORM = 1 << 2
FLAG_ETA_CLAMP = 1 << 3
FLAG_SANITIZE_NONFINITE = 1 << 4
FLAG_WEIGHTS_STATIC = 1 << 5
FLAG_INPUTS_READY = 1 << 6
# packed-code layouts (flag bits 7-8): Foundry's (default), Hetman-2b "Format 0" and "Format 1"
ENC_FOUNDRY = 0 << 7
ENC_FORMAT0 = 1 << 7
ENC_FORMAT1 = 2 << 7
ENC_MASK = 3 << 7
FLAG_ACCUMULATE = 1 << 9  # tq_ternary_backward_input: dX += result
FLAG_SHARED_INPUT = 1 << 10  # tq_bitlinear_grouped: one activation batch for all layers
FLAG_NORM_TOPK = 1 << 11  # tq_moe_swiglu: a token's weights add up to 1
FLAG_FP8_SQUARE = 1 << 12  # tq_quantize_fp8: 128 x 128 blocks
FLAG_FP8_W_ROWS = 1 << 13  # tq_fp8_gemm: w has a scale per row and block
FLAG_BF16_INPUT = 1 << 14  # tq_quantize_fp8: x is bf16
FLAG_BF16_OUTPUT = 1 << 15  # tq_fp8_gemm: y is bf16

STATUS = {0: "TQ_OK", 1: "TQ_ERR_NULL", 2: "TQ_ERR_SHAPE", 3: "TQ_ERR_ALIGN", 4: "TQ_ERR_ARG",
          5: "TQ_ERR_CUDA", 6: "TQ_ERR_DEVICE", 7: "TQ_ERR_TIMEOUT"}

# Entry points declared in include/tq.h, with their ctypes signatures.
_P, _I64, _U, _F, _I, _SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint, ctypes.c_float,
                              ctypes.c_int, ctypes.c_size_t)
SIGNATURES = {
    "tq_quantize_ternary_pack": (_I, [_P, _I64, _I64, _U, _P, _P, _P, _SZ, _P]),
    "tq_pack_workspace_bytes": (_SZ, [_I64, _I64, _U]),
    "tq_quantize_ternary_pack_threshold": (_I, [_P, _I64, _I64, _U, _F, _P, _P, _P, _SZ, _P]),
    "tq_quantize_ternary_pack_noalloc": (_I, [_P, _I64, _I64, _U, _P, _P, _P]),
    "tq_quantize_ternary_pack_abs_threshold": (_I, [_P, _I64, _I64, _U, _F, _P, _P, _P]),
    "tq_quantize_act_int8": (_I, [_P, _I64, _I64, _U, _F, _F, _P, _P, _P, _P]),
    "tq_fwht512": (_I, [_P, _P, _I64, _I64, _I, _P]),
    "tq_fwht_roundtrip": (_I, [_P, _P, _I64, _I64, _F, _F, _P, _P]),
    "tq_ternary_gemm": (_I, [_P, _P, _P, _P, _P, _U, _I64, _I64, _I64, _P, _P, _P]),
    "tq_ternary_gemm_ex": (_I, [_P, _P, _P, _P, _P, _U, _I64, _I64, _I64, _P, _P, _I, _P, _P, _P]),
    "tq_bitlinear_fused": (_I, [_P, _P, _F, _F, _F, _U, _P, _P, _I64, _I64, _I64, _P, _P, _P,
                                _P, _SZ, _P]),
    "tq_fused_workspace_bytes": (_SZ, [_I64, _I64, _U]),
    "tq_swiglu_mlp": (_I, [_P, _I64, _I64, _I64, _U, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "tq_swiglu_workspace_bytes": (_SZ, [_I64, _I64, _I64, _U]),
    "tq_bitlinear_grouped": (_I, [_P, _I64, _P, _P, _U, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "tq_grouped_workspace_bytes": (_SZ, [_I64, _I64, _I64, _U]),
    "tq_moe_swiglu": (_I, [_P, _I64, _I64, _I64, _I64, _I64, _U, _F, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ,
                           _P]),
    "tq_moe_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _I64, _U]),
    "tq_quantize_fp8": (_I, [_P, _I64, _I64, _U, _P, _F, _P, _P, _P, _P, _P]),
    "tq_fp8_row_bytes": (_SZ, [_I64]),
    "tq_fp8_gemm": (_I, [_P, _P, _P, _P, _U, _I64, _I64, _I64, _P, _P]),
    "tq_ternary_backward_input": (_I, [_P, _P, _P, _P, _U, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "tq_backward_input_workspace_bytes": (_SZ, [_I64, _I64]),
    "tq_ste_backward": (_I, [_P, _P, _P, _I64, _I64, _F, _U, _P, _P]),
    "tq_ternary_stochastic_flip": (_I, [_P, _P, _I64, _I64, _F, ctypes.POINTER(ctypes.c_uint64), _U, _P]),
    "tq_seed": (None, [ctypes.POINTER(ctypes.c_uint64), ctypes.c_uint64]),
    "tq_get_device_status": (_I, [_P]),
    "tq_selftest_wait_timeout": (_I, [ctypes.c_uint64, _I, _P]),
    "tq_status_string": (ctypes.c_char_p, [_I]),
    "tq_version": (_I, []),
}

_lib = None


class TqError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        msg = _lib.tq_status_string(code).decode() if _lib is not None else ""
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({msg})")


def load():
    """Load libtq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libtq.so not built ({LIB_PATH}); run "
                               "`python -m ternary_bit_linear_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, code: int):
    if code != 0:
        raise TqError(fn, code)


def _need(t, dtype, shape, name):
    if t is None:
        return
    if not t.is_cuda or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


# ---------------------------------------------------------------------------
# Raw C-ABI calls (tensors in, status checked); the caller owns every buffer.
# ---------------------------------------------------------------------------

def pack_workspace_bytes(N: int, K: int, flags: int) -> int:
    return load().tq_pack_workspace_bytes(N, K, flags)


def fused_workspace_bytes(M: int, K: int, flags: int) -> int:
    return load().tq_fused_workspace_bytes(M, K, flags)


def quantize_ternary_pack_(w, flags, packed, gamma, workspace=None, stream=None):
    import torch

    N, K = w.shape
    _need(w, torch.float32, (N, K), "w")
    _need(packed, torch.uint8, (N, K // 4), "packed")
    _need(gamma, torch.float32, (N if flags & GAMMA_PER_ROW else 1,), "gamma")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("tq_quantize_ternary_pack",
           load().tq_quantize_ternary_pack(_ptr(w), N, K, flags, _ptr(packed), _ptr(gamma),
                                           _ptr(workspace), ws_bytes, _stream(stream)))


def quantize_ternary_pack_threshold_(w, flags, ratio, packed, gamma, workspace=None, stream=None):
    import torch

    N, K = w.shape
    _need(w, torch.float32, (N, K), "w")
    _need(packed, torch.uint8, (N, K // 4), "packed")
    _need(gamma, torch.float32, (N if flags & GAMMA_PER_ROW else 1,), "gamma")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("tq_quantize_ternary_pack_threshold",
           load().tq_quantize_ternary_pack_threshold(_ptr(w), N, K, flags, float(ratio), _ptr(packed),
                                                     _ptr(gamma), _ptr(workspace), ws_bytes,
                                                     _stream(stream)))


def quantize_ternary_pack_abs_threshold_(w, flags, threshold, packed, gamma, stream=None):
    import torch

    N, K = w.shape
    _need(w, torch.float32, (N, K), "w")
    _need(packed, torch.uint8, (N, K // 4), "packed")
    _need(gamma, torch.float32, (1,), "gamma")
    _check("tq_quantize_ternary_pack_abs_threshold",
           load().tq_quantize_ternary_pack_abs_threshold(_ptr(w), N, K, flags, float(threshold), _ptr(packed),
                                                         _ptr(gamma), _stream(stream)))


def quantize_act_int8_(x, flags, eta_min, eta_max, xq, s_x, rowsum, stream=None):
    import torch

    M, K = x.shape
    _need(x, torch.float32, (M, K), "x")
    _need(xq, torch.int8, (M, K), "xq")
    _need(s_x, torch.float32, (M,), "s_x")
    _need(rowsum, torch.int32, (M,), "rowsum")
    _check("tq_quantize_act_int8",
           load().tq_quantize_act_int8(_ptr(x), M, K, flags, eta_min, eta_max, _ptr(xq),
                                       _ptr(s_x), _ptr(rowsum), _stream(stream)))


def fwht512_(x, y, normalize=True, stream=None):
    import torch

    rows, K = x.shape
    _need(x, torch.float32, (rows, K), "x")
    _need(y, torch.float32, (rows, K), "y")
    _check("tq_fwht512", load().tq_fwht512(_ptr(x), _ptr(y), rows, K, int(bool(normalize)),
                                           _stream(stream)))


def ternary_gemm_(xq, s_x, rowsum, packed, gamma, flags, y, acc=None, stream=None):
    import torch

    M, K = xq.shape
    N = packed.shape[0]
    _need(xq, torch.int8, (M, K), "xq")
    _need(packed, torch.uint8, (N, K // 4), "packed")
    _need(y, torch.float32, (M, N), "y")
    _need(acc, torch.int32, (M, N), "acc")
    _check("tq_ternary_gemm",
           load().tq_ternary_gemm(_ptr(xq), _ptr(s_x), _ptr(rowsum), _ptr(packed), _ptr(gamma),
                                  flags, M, N, K, _ptr(y), _ptr(acc), _stream(stream)))


def ternary_gemm_ex_(xq, s_x, rowsum, packed, gamma, flags, y, acc=None, bias=None, acc_bias=None,
                     out_shift=0, stream=None):
    import torch

    M, K = xq.shape
    N = packed.shape[0]
    _need(xq, torch.int8, (M, K), "xq")
    _need(packed, torch.uint8, (N, K // 4), "packed")
    _need(y, torch.float32, (M, N), "y")
    _need(acc, torch.int32, (M, N), "acc")
    _need(bias, torch.float32, (N,), "bias")
    _need(acc_bias, torch.int32, (N,), "acc_bias")
    _check("tq_ternary_gemm_ex",
           load().tq_ternary_gemm_ex(_ptr(xq), _ptr(s_x), _ptr(rowsum), _ptr(packed), _ptr(gamma), flags, M, N, K,
                                     _ptr(bias), _ptr(acc_bias), int(out_shift), _ptr(y), _ptr(acc),
                                     _stream(stream)))


def bitlinear_fused_(x, packed, gamma, flags, y, workspace, rms_gain=None, rms_eps=1e-6,
                     eta_min=0.05, eta_max=40.0, xq_out=None, s_x_out=None, stream=None):
    import torch

    M, K = x.shape
    N = packed.shape[0]
    _need(x, torch.float32, (M, K), "x")
    _need(y, torch.float32, (M, N), "y")
    _check("tq_bitlinear_fused",
           load().tq_bitlinear_fused(_ptr(x), _ptr(rms_gain), rms_eps, eta_min, eta_max, flags,
                                     _ptr(packed), _ptr(gamma), M, N, K, _ptr(y), _ptr(xq_out),
                                     _ptr(s_x_out), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _stream(stream)))


def fwht_roundtrip_(x, y, eta_min=0.05, eta_max=40.0, eta_out=None, stream=None):
    import torch

    rows, K = x.shape
    _need(x, torch.float32, (rows, K), "x")
    _need(y, torch.float32, (rows, K), "y")
    _need(eta_out, torch.float32, (rows,), "eta_out")
    _check("tq_fwht_roundtrip",
           load().tq_fwht_roundtrip(_ptr(x), _ptr(y), rows, K, float(eta_min), float(eta_max), _ptr(eta_out),
                                    _stream(stream)))


def swiglu_workspace_bytes(M: int, d_model: int, d_ffn: int, flags: int) -> int:
    return int(load().tq_swiglu_workspace_bytes(M, d_model, d_ffn, flags))


def grouped_workspace_bytes(G: int, M: int, K: int, flags: int) -> int:
    return int(load().tq_grouped_workspace_bytes(G, M, K, flags))


def bitlinear_grouped_(x, packed, gamma, flags, y, workspace, stream=None):
    """G same-shape layers: x [G, M, K] (or [M, K] with FLAG_SHARED_INPUT),
    packed / gamma: sequences of G device tensors, y [G, M, N]."""
    import torch

    G = len(packed)
    if len(gamma) != G:
        raise ValueError("packed and gamma must have one entry per layer")
    M, K = x.shape[-2], x.shape[-1]
    N = packed[0].shape[0]
    _need(x, torch.float32, (M, K) if flags & FLAG_SHARED_INPUT else (G, M, K), "x")
    _need(y, torch.float32, (G, M, N), "y")
    for p in packed:
        _need(p, torch.uint8, (N, K // 4), "packed")
    arr = ctypes.c_void_p * G
    pp = arr(*[p.data_ptr() for p in packed])
    gp = arr(*[g.data_ptr() for g in gamma])
    _check("tq_bitlinear_grouped",
           load().tq_bitlinear_grouped(_ptr(x), G, ctypes.cast(pp, ctypes.c_void_p), ctypes.cast(gp, ctypes.c_void_p),
                                       flags, M, N, K, _ptr(y), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))


def grouped_intermediates(workspace, G: int, M: int, K: int, flags: int) -> dict:
    """x_q (back in plain [Gx, M, K] order), s_x and rowsum from the
    workspace of tq_bitlinear_grouped (the layout the header states)."""
    import torch

    Gx = 1 if flags & FLAG_SHARED_INPUT else G
    al = lambda b: (b + 255) & ~255
    o1 = al(Gx * M * K)
    o2 = o1 + al(Gx * M * 4)
    raw = workspace[:Gx * M * K].view(Gx * M, K // 16, 4, 4)
    c = torch.arange(K // 16, device=workspace.device)
    pos = c ^ (2 * ((c >> 3) & 1))
    xq = raw[:, pos].transpose(2, 3).reshape(Gx, M, K).view(torch.int8)
    sx = workspace[o1:o1 + Gx * M * 4].view(torch.float32).view(Gx, M)
    rs = workspace[o2:o2 + Gx * M * 4].view(torch.int32).view(Gx, M)
    return {"xq": xq, "s_x": sx, "rowsum": rs}


def swiglu_intermediates(workspace, M: int, d_model: int, d_ffn: int) -> dict:
    """Views of what tq_swiglu_mlp leaves in its workspace (the layout the
    header states: eight parts, each starting on a 256-byte boundary)."""
    import torch

    sizes = [(M * d_model, torch.int8, (M, d_model), "xq1"), (M, torch.float32, (M,), "s_x1"),
             (M, torch.int32, (M,), "rowsum1"), (M * d_ffn, torch.float32, (M, d_ffn), "y_gate"),
             (M * d_ffn, torch.float32, (M, d_ffn), "y_up"), (M * d_ffn, torch.int8, (M, d_ffn), "xq2"),
             (M, torch.float32, (M,), "s_x2"), (M, torch.int32, (M,), "rowsum2")]
    out, off = {}, 0
    for n, dt, shape, name in sizes:
        nb = n * torch.tensor([], dtype=dt).element_size()
        out[name] = workspace[off:off + nb].view(dt).view(shape)
        off += (nb + 255) & ~255
    if off > workspace.numel():
        raise ValueError("workspace smaller than tq_swiglu_workspace_bytes")
    return out


def swiglu_mlp_(x, gate, up, down, flags, y, workspace, clamp_val=10.0, act_out=None, stream=None):
    """gate, up, down: (packed, gamma) pairs."""
    import torch

    M, D = x.shape
    F = gate[0].shape[0]
    _need(x, torch.float32, (M, D), "x")
    _need(y, torch.float32, (M, D), "y")
    _need(act_out, torch.float32, (M, F), "act_out")
    _need(gate[0], torch.uint8, (F, D // 4), "gate packed")
    _need(up[0], torch.uint8, (F, D // 4), "up packed")
    _need(down[0], torch.uint8, (D, F // 4), "down packed")
    _check("tq_swiglu_mlp",
           load().tq_swiglu_mlp(_ptr(x), M, D, F, flags, float(clamp_val), _ptr(gate[0]), _ptr(gate[1]),
                                _ptr(up[0]), _ptr(up[1]), _ptr(down[0]), _ptr(down[1]), _ptr(y), _ptr(act_out),
                                _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def fp8_row_bytes(K: int) -> int:
    """Bytes of a row of K e4m3 codes: K rounded up to 16."""
    return (K + 15) // 16 * 16


def _fit(t, dtype, shape, dev, name):
    """The check of _need for calls that last a few microseconds; `dev` is the index of
    the CUDA device of all tensors of the call.  Returns the address."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on cuda:{dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _call(fn, dev, stream, *args):
    """The C call on device `dev`: on `stream`, or on that device's current stream."""
    import torch

    if dev < 0:
        raise ValueError(f"{fn}: expected CUDA tensors")
    f = getattr(_lib or load(), fn)
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        code = f(*args, s)
    else:
        with torch.cuda.device(dev):
            code = f(*args, s)
    if code != 0:
        raise TqError(fn, code)


def moe_workspace_bytes(M: int, d_model: int, d_ffn: int, n_experts: int, top_k: int, flags: int) -> int:
    return load().tq_moe_workspace_bytes(M, d_model, d_ffn, n_experts, top_k, flags)


def moe_swiglu_(x, router, gate, up, down, flags, y, ids, weights, workspace, clamp_val=10.0, stream=None):
    """gate, up, down: (packed, gamma) pairs, the experts stacked along the first
    dimension; router [E, D] float32, or None: ids [M, k] int32 and weights [M, k]
    float32 are then read (an id outside [0, E): no expert) instead of written."""
    import torch

    M, D = x.shape
    E, F = gate[0].shape[0], gate[0].shape[1]
    k = ids.shape[1]
    dev, f32, u8 = x.get_device(), torch.float32, torch.uint8
    gf, gd = ((E, F), (E, D)) if flags & GAMMA_PER_ROW else ((E,), (E,))
    _call("tq_moe_swiglu", dev, stream, _fit(x, f32, (M, D), dev, "x"), M, D, F, E, k, flags, clamp_val,
          None if router is None else _fit(router, f32, (E, D), dev, "router"),
          _fit(gate[0], u8, (E, F, D // 4), dev, "gate packed"), _fit(gate[1], f32, gf, dev, "gate gamma"),
          _fit(up[0], u8, (E, F, D // 4), dev, "up packed"), _fit(up[1], f32, gf, dev, "up gamma"),
          _fit(down[0], u8, (E, D, F // 4), dev, "down packed"), _fit(down[1], f32, gd, dev, "down gamma"),
          _fit(y, f32, (M, D), dev, "y"), _fit(ids, torch.int32, (M, k), dev, "ids"),
          _fit(weights, f32, (M, k), dev, "weights"),
          _fit(workspace, u8, (workspace.numel(),), dev, "workspace"), workspace.numel())


def quantize_fp8_(x, flags, q, s, qt=None, st=None, rms_gain=None, rms_eps=1e-6, stream=None):
    """x [R, C] float32 (bfloat16 with FLAG_BF16_INPUT); q [R, fp8_row_bytes(C)]
    float8_e4m3fn; s [ceil(C/128), R], or [ceil(R/128), ceil(C/128)] with
    FLAG_FP8_SQUARE; qt, st: the same for the transpose of x, or None."""
    import torch

    R, C = x.shape
    rb, cb = -(-R // 128), -(-C // 128)
    square, dev, f8, f32 = flags & FLAG_FP8_SQUARE, x.get_device(), torch.float8_e4m3fn, torch.float32
    _call("tq_quantize_fp8", dev, stream,
          _fit(x, torch.bfloat16 if flags & FLAG_BF16_INPUT else f32, (R, C), dev, "x"), R, C, flags,
          None if rms_gain is None else _fit(rms_gain, f32, (C,), dev, "rms_gain"), rms_eps,
          _fit(q, f8, (R, (C + 15) // 16 * 16), dev, "q"),
          _fit(s, f32, (rb, cb) if square else (cb, R), dev, "s"),
          None if qt is None else _fit(qt, f8, (C, (R + 15) // 16 * 16), dev, "qt"),
          None if st is None else _fit(st, f32, (cb, rb) if square else (rb, C), dev, "st"))


def fp8_gemm_(xq, s_x, wq, s_w, K, flags, y, stream=None):
    """xq [M, fp8_row_bytes(K)], wq [N, fp8_row_bytes(K)] float8_e4m3fn; s_x
    [ceil(K/128), M]; s_w [ceil(N/128), ceil(K/128)], or [ceil(K/128), N] with
    FLAG_FP8_W_ROWS; y [M, N] float32, or bfloat16 with FLAG_BF16_OUTPUT."""
    import torch

    M, N, ld, kb = xq.shape[0], wq.shape[0], (K + 15) // 16 * 16, -(-K // 128)
    dev, f8, f32 = xq.get_device(), torch.float8_e4m3fn, torch.float32
    _call("tq_fp8_gemm", dev, stream, _fit(xq, f8, (M, ld), dev, "xq"), _fit(s_x, f32, (kb, M), dev, "s_x"),
          _fit(wq, f8, (N, ld), dev, "wq"),
          _fit(s_w, f32, (kb, N) if flags & FLAG_FP8_W_ROWS else (-(-N // 128), kb), dev, "s_w"), flags, M, N, K,
          _fit(y, torch.bfloat16 if flags & FLAG_BF16_OUTPUT else f32, (M, N), dev, "y"))


def backward_input_workspace_bytes(M: int, N: int) -> int:
    return load().tq_backward_input_workspace_bytes(M, N)


def ternary_backward_input_(dY, packed, gamma, flags, dX, workspace, row_scale=None, stream=None):
    import torch

    M, N = dY.shape
    K = packed.shape[1] * 4
    _need(dY, torch.float32, (M, N), "dY")
    _need(packed, torch.uint8, (N, K // 4), "packed")
    _need(gamma, torch.float32, (N if flags & GAMMA_PER_ROW else 1,), "gamma")
    _need(row_scale, torch.float32, (M,), "row_scale")
    _need(dX, torch.float32, (M, K), "dX")
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("tq_ternary_backward_input",
           load().tq_ternary_backward_input(_ptr(dY), _ptr(packed), _ptr(gamma), _ptr(row_scale), flags, M, N, K,
                                            _ptr(dX), _ptr(workspace), ws_bytes, _stream(stream)))


def ste_backward_(grad, w, gamma, flags, out, tau=1.0, stream=None):
    import torch

    N, K = w.shape
    _need(grad, torch.float32, (N, K), "grad")
    _need(w, torch.float32, (N, K), "w")
    _need(gamma, torch.float32, (N if flags & GAMMA_PER_ROW else 1,), "gamma")
    _need(out, torch.float32, (N, K), "out")
    _check("tq_ste_backward", load().tq_ste_backward(_ptr(grad), _ptr(w), _ptr(gamma), N, K, float(tau), flags,
                                                     _ptr(out), _stream(stream)))


def seed(value: int) -> int:
    """fq_seed: the xorshift64 state for `value`."""
    st = ctypes.c_uint64(0)
    load().tq_seed(ctypes.byref(st), ctypes.c_uint64(value))
    return st.value


def ternary_stochastic_flip_(packed, grad, temperature, state: int, flags=0, stream=None) -> int:
    """Flips `packed` in place; returns the generator state after the N*K draws."""
    import torch

    N, K = grad.shape
    _need(grad, torch.float32, (N, K), "grad")
    _need(packed, torch.uint8, (N, K // 4), "packed")
    st = ctypes.c_uint64(state)
    _check("tq_ternary_stochastic_flip",
           load().tq_ternary_stochastic_flip(_ptr(packed), _ptr(grad), N, K, float(temperature), ctypes.byref(st),
                                             flags, _stream(stream)))
    return st.value


def device_status(stream=None) -> int:
    """Synchronises the stream; returns and clears the device status word."""
    return load().tq_get_device_status(_stream(stream))


def selftest_wait_timeout(limit_ns: int, sleeping: bool = False, stream=None):
    """Launch the bounded-wait self-test (a wait that nothing completes, given
    up after limit_ns); the next device_status() reports TQ_ERR_TIMEOUT."""
    _check("tq_selftest_wait_timeout",
           load().tq_selftest_wait_timeout(int(limit_ns), int(bool(sleeping)), _stream(stream)))


# ---------------------------------------------------------------------------
# Allocating conveniences (torch allocates; the kernels compute).  With `stream`
# the work runs there and the buffers are taken there; as for every call, the
# inputs must be complete on that stream, and whoever reads the results on
# another one waits for it.
# ---------------------------------------------------------------------------

def _under(stream, call, first, *args):
    """`call` with `stream` current: its buffers then come from that stream's pool, so scratch
    dropped on return is reused behind the kernels that work on it, and nothing that another
    stream still works on is written.  The results are tied to the caller's stream too: what
    it frees goes back once its own work is done."""
    import torch

    if first.device != stream.device:
        raise ValueError(f"stream on {stream.device}, tensors on {first.device}")
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = call(first, *args)
    for t in out if isinstance(out, tuple) else (out,):
        t.record_stream(here)
    return out


def quantize_ternary_pack(w, per_row: bool, sanitize: bool = False, stream=None):
    import torch

    if stream is not None:
        return _under(stream, quantize_ternary_pack, w, per_row, sanitize)
    N, K = w.shape
    flags = (GAMMA_PER_ROW if per_row else 0) | (FLAG_SANITIZE_NONFINITE if sanitize else 0)
    packed = torch.empty((N, K // 4), dtype=torch.uint8, device=w.device)
    gamma = torch.empty((N if per_row else 1,), dtype=torch.float32, device=w.device)
    nws = pack_workspace_bytes(N, K, flags)
    ws = torch.empty((max(nws, 16),), dtype=torch.uint8, device=w.device) if nws else None
    quantize_ternary_pack_(w, flags, packed, gamma, ws)
    return packed, gamma


def quantize_act_int8(x, clamp_eta: bool = False, eta_min: float = 0.05, eta_max: float = 40.0,
                      sanitize: bool = False, stream=None):
    import torch

    if stream is not None:
        return _under(stream, quantize_act_int8, x, clamp_eta, eta_min, eta_max, sanitize)
    M, K = x.shape
    flags = (FLAG_ETA_CLAMP if clamp_eta else 0) | (FLAG_SANITIZE_NONFINITE if sanitize else 0)
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s_x = torch.empty((M,), dtype=torch.float32, device=x.device)
    rowsum = torch.empty((M,), dtype=torch.int32, device=x.device)
    quantize_act_int8_(x, flags, eta_min, eta_max, xq, s_x, rowsum)
    return xq, s_x, rowsum


def fwht512(x, normalize: bool = True, stream=None):
    import torch

    if stream is not None:
        return _under(stream, fwht512, x, normalize)
    y = torch.empty_like(x)
    fwht512_(x, y, normalize)
    return y


def ternary_gemm(xq, s_x, rowsum, packed, gamma, per_row: bool, with_acc: bool = False,
                 stream=None):
    import torch

    if stream is not None:
        return _under(stream, ternary_gemm, xq, s_x, rowsum, packed, gamma, per_row, with_acc)
    M, N = xq.shape[0], packed.shape[0]
    y = torch.empty((M, N), dtype=torch.float32, device=xq.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=xq.device) if with_acc else None
    ternary_gemm_(xq, s_x, rowsum, packed, gamma, GAMMA_PER_ROW if per_row else 0, y, acc)
    return (y, acc) if with_acc else y


def bitlinear_fused(x, packed, gamma, per_row: bool, rmsnorm: bool = True, fwht: bool = True,
                    rms_gain=None, rms_eps: float = 1e-6, clamp_eta: bool = False,
                    eta_min: float = 0.05, eta_max: float = 40.0, sanitize: bool = False,
                    return_xq: bool = False, stream=None):
    import torch

    if stream is not None:
        return _under(stream, bitlinear_fused, x, packed, gamma, per_row, rmsnorm, fwht, rms_gain, rms_eps,
                      clamp_eta, eta_min, eta_max, sanitize, return_xq)
    M, K = x.shape
    N = packed.shape[0]
    flags = ((GAMMA_PER_ROW if per_row else 0) | (FLAG_RMSNORM if rmsnorm else 0) |
             (FLAG_FWHT if fwht else 0) | (FLAG_ETA_CLAMP if clamp_eta else 0) |
             (FLAG_SANITIZE_NONFINITE if sanitize else 0))
    y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    ws = torch.empty((fused_workspace_bytes(M, K, flags),), dtype=torch.uint8, device=x.device)
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device) if return_xq else None
    sx = torch.empty((M,), dtype=torch.float32, device=x.device) if return_xq else None
    bitlinear_fused_(x, packed, gamma, flags, y, ws, rms_gain, rms_eps, eta_min, eta_max, xq, sx)
    return (y, xq, sx) if return_xq else y


def moe_swiglu(x, router, gate, up, down, top_k: int, per_row: bool = False, rmsnorm: bool = True,
               norm_topk: bool = True, sanitize: bool = False, clamp_val: float = 10.0, stream=None):
    """A mixture-of-experts layer for up to 64 tokens: (y, ids, weights)."""
    import torch

    if stream is not None:
        return _under(stream, moe_swiglu, x, router, gate, up, down, top_k, per_row, rmsnorm, norm_topk, sanitize, clamp_val)
    M, D = x.shape
    E, F = gate[0].shape[0], gate[0].shape[1]
    flags = (FLAG_FWHT | (GAMMA_PER_ROW if per_row else 0) | (FLAG_RMSNORM if rmsnorm else 0) |
             (FLAG_NORM_TOPK if norm_topk else 0) | (FLAG_SANITIZE_NONFINITE if sanitize else 0))
    y = torch.empty_like(x)
    ids = x.new_empty((M, top_k), dtype=torch.int32)
    weights = x.new_empty((M, top_k))
    ws = x.new_empty((moe_workspace_bytes(M, D, F, E, top_k, flags),), dtype=torch.uint8)
    moe_swiglu_(x, router, gate, up, down, flags, y, ids, weights, ws, clamp_val)
    return y, ids, weights


def _new(shape, dtype, device):
    """torch.empty of two dimensions (the strided form costs about half as much)."""
    import torch

    return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)


def quantize_fp8(x, square: bool = False, transpose: bool = False, rmsnorm: bool = False, rms_gain=None,
                 rms_eps: float = 1e-6, stream=None):
    """(q, s) of x [R, C] (float32 or bfloat16), or (q, s, qt, st) with `transpose`."""
    import torch

    if stream is not None:
        return _under(stream, quantize_fp8, x, square, transpose, rmsnorm, rms_gain, rms_eps)
    R, C = x.shape
    rb, cb, ldq, ldt = (R + 127) // 128, (C + 127) // 128, (C + 15) // 16 * 16, (R + 15) // 16 * 16
    dev, f8, f32, bf16 = x.get_device(), torch.float8_e4m3fn, torch.float32, x.dtype is torch.bfloat16
    flags = ((FLAG_FP8_SQUARE if square else 0) | (FLAG_RMSNORM if rmsnorm else 0) | (FLAG_BF16_INPUT if bf16 else 0))
    q = _new((R, ldq), f8, x.device)
    s = _new((rb, cb) if square else (cb, R), f32, x.device)
    qt = st = None
    if transpose:
        qt = _new((C, ldt), f8, x.device)
        st = _new((cb, rb) if square else (rb, C), f32, x.device)
    _call("tq_quantize_fp8", dev, None, _fit(x, torch.bfloat16 if bf16 else f32, (R, C), dev, "x"), R, C, flags,
          None if rms_gain is None else _fit(rms_gain, f32, (C,), dev, "rms_gain"), rms_eps, q.data_ptr(), s.data_ptr(),
          qt.data_ptr() if transpose else None, st.data_ptr() if transpose else None)
    return (q, s, qt, st) if transpose else (q, s)


def fp8_gemm(xq, s_x, wq, s_w, K: int, w_rows: bool = False, bf16: bool = False, stream=None):
    """y [M, N] of codes and scales as quantize_fp8 gives them (w: its square form, or with `w_rows` its row form)."""
    import torch

    if stream is not None:
        return _under(stream, fp8_gemm, xq, s_x, wq, s_w, K, w_rows, bf16)
    y = _new((xq.shape[0], wq.shape[0]), torch.bfloat16 if bf16 else torch.float32, xq.device)
    fp8_gemm_(xq, s_x, wq, s_w, K, (FLAG_FP8_W_ROWS if w_rows else 0) | (FLAG_BF16_OUTPUT if bf16 else 0), y)
    return y
