"""Refusals of the mixture-of-experts layer, on fake pointers that are never dereferenced: every check comes before
any device work."""
import ctypes

import pytest

import ternary_bit_linear_b200 as tq
from ternary_bit_linear_b200 import build as tqbuild

NULL, SHAPE, ALIGN, ARG = 1, 2, 3, 4
M, D, F, E, K = 5, 512, 1024, 6, 3
FL = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW


@pytest.fixture(scope="module")
def lib():
    tqbuild.build()
    return tq.load()


def P(mib, off=0):
    return ctypes.c_void_p(0x10000000 + (mib << 20) + off)


def caller(lib):
    names = ["x", "M", "D", "F", "E", "k", "flags", "clamp", "router", "gp", "gg", "up", "ug", "dp", "dg", "y", "ids",
             "w", "ws", "wsb", "stream"]
    ok = [P(0), M, D, F, E, K, FL, 10.0, P(1), P(2), P(4), P(6), P(8), P(10), P(12), P(14), P(15), P(16), P(18),
          lib.tq_moe_workspace_bytes(M, D, F, E, K, FL), None]

    def call(**kw):
        assert set(kw) <= set(names)
        return lib.tq_moe_swiglu(*[kw.get(n, v) for n, v in zip(names, ok)])
    return call


BAD_SHAPES = [("M", 0), ("M", -1), ("M", 65), ("D", 0), ("D", 500), ("D", 8704), ("F", 0), ("F", 640), ("F", 8704),
              ("E", 0), ("E", 257), ("k", 0), ("k", 7), ("k", 17)]


@pytest.mark.parametrize("name,value", BAD_SHAPES)
def test_shapes(lib, name, value):
    assert caller(lib)(**{name: value}) == SHAPE
    shape = dict(M=M, D=D, F=F, E=E, k=K)
    shape[name] = value
    assert lib.tq_moe_workspace_bytes(*shape.values(), FL) == 0


def test_pointers(lib):
    call = caller(lib)
    for name in ("x", "gp", "gg", "up", "ug", "dp", "dg", "y", "ids", "w", "ws"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: P(40, 8)}) == ALIGN, name
    assert call(router=P(40, 4)) == ALIGN


def test_arguments(lib):
    call = caller(lib)
    for flags in (FL & ~tq.FLAG_FWHT, FL | tq.FLAG_INPUTS_READY, FL | tq.FLAG_ACCUMULATE, FL | tq.ENC_MASK, FL | 1 << 20):
        assert call(flags=flags) == ARG
    assert call(router=None, flags=FL | tq.FLAG_NORM_TOPK) == ARG   # given weights are used as they are
    for clamp in (0.0, -1.0, float("nan"), float("inf")):
        assert call(clamp=clamp) == ARG
    need = lib.tq_moe_workspace_bytes(M, D, F, E, K, FL)
    assert need >= M * (D + 4 * E) + M * K * (5 * F + 4 * D)
    assert call(wsb=need - 1) == ARG


def test_overlaps(lib):
    call = caller(lib)
    assert call(y=P(0, M * D * 4 - 16)) == ARG                       # x
    assert call(y=P(1, E * D * 4 - 16)) == ARG                       # router
    assert call(ws=P(2, E * F * D // 4 - 16)) == ARG                 # gate
    assert call(w=P(12, E * D * 4 - 16)) == ARG                      # down gamma
    assert call(ids=P(16)) == ARG                                    # ids on weights
    assert call(w=P(14, 16)) == ARG                                  # weights on y
    assert call(y=P(18, 512)) == ARG                                 # y in the workspace


def test_binding_checks_tensors():
    import torch
    x = torch.zeros(2, 512)
    pack = (torch.zeros(2, 512, 128, dtype=torch.uint8), torch.zeros(2))
    with pytest.raises(ValueError):   # no CPU path
        tq.moe_swiglu(x, torch.zeros(2, 512), pack, pack, pack, 1)


@pytest.mark.parametrize("name,value", BAD_SHAPES)
def test_a_refused_shape_is_named_whatever_its_buffers(lib, name, value):
    """The scratch of a refused shape has 0 bytes and no address; empty tensors have none either."""
    call = caller(lib)
    assert call(**{name: value}, ws=None, wsb=0) == SHAPE
    assert call(**{name: value}, ws=None, wsb=0, x=None, y=None, ids=None, w=None) == SHAPE
