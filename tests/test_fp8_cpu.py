"""Refusals of the block-scaled e4m3 entry points, on fake pointers that are never dereferenced: every check comes
before any device work."""
import ctypes

import pytest

import ternary_bit_linear_b200 as tq
from ternary_bit_linear_b200 import build as tqbuild

NULL, SHAPE, ALIGN, ARG = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    tqbuild.build()
    return tq.load()


def P(mib, off=0):
    return ctypes.c_void_p(0x10000000 + (mib << 20) + off)


def caller(f, names, ok):
    def call(**kw):
        assert set(kw) <= set(names)
        return f(*[kw.get(n, v) for n, v in zip(names, ok)])
    return call


def test_flags_are_their_own_bits():
    new = [tq.FLAG_NORM_TOPK, tq.FLAG_FP8_SQUARE, tq.FLAG_FP8_W_ROWS, tq.FLAG_BF16_INPUT, tq.FLAG_BF16_OUTPUT]
    old = [tq.GAMMA_PER_ROW, tq.FLAG_FWHT, tq.FLAG_RMSNORM, tq.FLAG_ETA_CLAMP, tq.FLAG_SANITIZE_NONFINITE,
           tq.FLAG_WEIGHTS_STATIC, tq.FLAG_INPUTS_READY, tq.FLAG_ACCUMULATE, tq.FLAG_SHARED_INPUT, tq.ENC_FORMAT0,
           tq.ENC_FORMAT1]
    assert len(set(new + old)) == len(new + old) and all(v & (v - 1) == 0 for v in new)


def test_row_bytes(lib):
    for k, want in ((-1, 0), (0, 0), (1, 16), (16, 16), (17, 32), (4096, 4096)):
        assert lib.tq_fp8_row_bytes(k) == want
        if k > 0:
            assert tq.fp8_row_bytes(k) == want


def test_quantize_refusals(lib):
    call = caller(lib.tq_quantize_fp8, ["x", "rows", "cols", "flags", "gain", "eps", "q", "s", "qt", "st", "stream"],
                  [P(0), 300, 200, 0, None, 1e-6, P(1), P(2), P(3), P(4), None])
    for name in ("x", "q", "s"):
        assert call(**{name: None}) == NULL
    assert call(qt=None) == NULL and call(st=None) == NULL      # one of the two alone
    for bad in (0, -1, (1 << 24) + 1):
        assert call(rows=bad) == SHAPE and call(cols=bad) == SHAPE
    for flags in (tq.GAMMA_PER_ROW, tq.FLAG_SANITIZE_NONFINITE, tq.FLAG_BF16_OUTPUT, 1 << 20):
        assert call(flags=flags) == ARG
    assert call(flags=tq.FLAG_RMSNORM) == ARG                   # with a transpose
    assert call(flags=tq.FLAG_RMSNORM | tq.FLAG_FP8_SQUARE, qt=None, st=None) == ARG
    assert call(gain=P(5)) == ARG                               # a gain without the norm
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(flags=tq.FLAG_RMSNORM, qt=None, st=None, eps=eps) == ARG
    for name in ("x", "q", "s", "qt", "st"):
        assert call(**{name: P(6, 8)}) == ALIGN
    assert call(flags=tq.FLAG_RMSNORM, qt=None, st=None, gain=P(6, 4)) == ALIGN
    assert call(q=P(0, 300 * 200 * 4 - 16)) == ARG              # over x's end
    assert call(st=P(1, 300 * 208 - 16)) == ARG                 # over the padded end of q
    assert call(qt=P(3), st=P(3, 200 * 304 - 16)) == ARG        # over the padded end of qt


def test_gemm_refusals(lib):
    M, N, K = 40, 300, 200
    call = caller(lib.tq_fp8_gemm, ["xq", "sx", "wq", "sw", "flags", "M", "N", "K", "y", "stream"],
                  [P(0), P(1), P(2), P(3), 0, M, N, K, P(4), None])
    for name in ("xq", "sx", "wq", "sw", "y"):
        assert call(**{name: None}) == NULL
        assert call(**{name: P(6, 8)}) == ALIGN
    for bad in (0, -5, (1 << 24) + 1):
        assert call(M=bad) == SHAPE and call(N=bad) == SHAPE and call(K=bad) == SHAPE
    for flags in (tq.GAMMA_PER_ROW, tq.FLAG_INPUTS_READY, tq.FLAG_BF16_INPUT, tq.FLAG_FP8_SQUARE,
                  tq.FLAG_BF16_OUTPUT | tq.FLAG_ACCUMULATE):
        assert call(flags=flags) == ARG
    assert call(y=P(0, M * 208 - 16)) == ARG                    # over the padded end of xq
    assert call(y=P(2, N * 208 - 16)) == ARG
    assert call(y=P(1, 2 * M * 4 - 16)) == ARG
    assert call(y=P(3, 16), flags=tq.FLAG_FP8_W_ROWS) == ARG
    assert call(y=P(3, 2 * N * 4 - 16), flags=tq.FLAG_FP8_W_ROWS) == ARG


def test_binding_checks_tensors():
    import torch
    x = torch.zeros(4, 32)
    with pytest.raises(ValueError):   # no CPU path
        tq.quantize_fp8(x)


def test_an_empty_matrix_is_a_refused_shape(lib):
    """Empty tensors have no address: the shape is what is wrong."""
    assert lib.tq_quantize_fp8(None, 0, 64, 0, None, 1e-6, None, None, None, None, None) == SHAPE
    assert lib.tq_quantize_fp8(None, 64, 0, 0, None, 1e-6, None, None, None, None, None) == SHAPE
    for shape in ((0, 64, 64), (64, 0, 64), (64, 64, 0)):
        assert lib.tq_fp8_gemm(None, None, None, None, 0, *shape, None, None) == SHAPE
