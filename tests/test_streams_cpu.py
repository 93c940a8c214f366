"""Where the allocating calls take their buffers when they are given a stream: from that stream, with it current, and
the results tied to the caller's stream too.  Shown on the CPU with stand-ins for torch's streams and the raw calls."""
import contextlib

import pytest
import torch

import ternary_bit_linear_b200 as tq
from ternary_bit_linear_b200 import build as tqbuild


class FakeStream:
    device = torch.device("cpu")
    cuda_stream = 0


def pack(n, k):
    return torch.zeros(n, k // 4, dtype=torch.uint8), torch.ones(n)


def experts(e, n, k):
    return torch.zeros(e, n, k // 4, dtype=torch.uint8), torch.ones(e)


CODES = torch.zeros(4, 512, dtype=torch.uint8)
CALLS = {  # call, the raw call it makes, how many results
    "quantize_ternary_pack": (lambda s: tq.quantize_ternary_pack(torch.ones(8, 512), False, stream=s), "quantize_ternary_pack_", 2),
    "quantize_act_int8": (lambda s: tq.quantize_act_int8(torch.ones(4, 512), stream=s), "quantize_act_int8_", 3),
    "fwht512": (lambda s: tq.fwht512(torch.ones(4, 512), stream=s), "fwht512_", 1),
    "ternary_gemm": (lambda s: tq.ternary_gemm(torch.zeros(4, 512, dtype=torch.int8), torch.ones(4), torch.ones(4), *pack(8, 512),
                                               True, True, stream=s), "ternary_gemm_", 2),
    "bitlinear_fused": (lambda s: tq.bitlinear_fused(torch.ones(4, 512), *pack(8, 512), True, return_xq=True, stream=s),
                        "bitlinear_fused_", 3),
    "moe_swiglu": (lambda s: tq.moe_swiglu(torch.ones(4, 512), torch.ones(2, 512), experts(2, 512, 512), experts(2, 512, 512),
                                           experts(2, 512, 512), 1, stream=s), "moe_swiglu_", 3),
    "quantize_fp8": (lambda s: tq.quantize_fp8(torch.ones(4, 512), stream=s), "_call", 2),
    "quantize_fp8 transposed": (lambda s: tq.quantize_fp8(torch.ones(4, 512), transpose=True, stream=s), "_call", 4),
    "fp8_gemm": (lambda s: tq.fp8_gemm(CODES, torch.ones(4, 4), CODES, torch.ones(1, 4), 512, stream=s), "fp8_gemm_", 1),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_belong_to_the_given_stream(monkeypatch, name):
    tqbuild.build()
    tq.load()
    call, raw, results = CALLS[name]
    side, here = FakeStream(), FakeStream()
    now, taken, launched, tied = [here], [], [], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def counting(make):
        def f(*a, **k):
            t = make(*a, **k)
            taken.append((t, now[-1]))
            return t
        return f

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    for owner, fn in ((torch, "empty"), (torch, "empty_like"), (torch, "empty_strided"), (torch.Tensor, "new_empty")):
        monkeypatch.setattr(owner, fn, counting(getattr(owner, fn)))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: tied.append((t.data_ptr(), s)))
    monkeypatch.setattr(tq, raw, lambda *a, **k: launched.append(now[-1]))
    out = call(side)
    out = out if isinstance(out, tuple) else (out,)
    assert len(out) == results
    assert len(taken) >= results and all(s is side for _, s in taken)
    assert launched == [side] and now == [here]
    assert sorted(p for p, s in tied if s is here) == sorted(t.data_ptr() for t in out)
    # without a stream: the current one, and nothing to tie
    del taken[:], launched[:], tied[:]
    call(None)
    assert launched == [here] and all(s is here for _, s in taken) and not tied


def test_stream_of_another_device():
    side = FakeStream()
    side.device = torch.device("cuda", 3)
    with pytest.raises(ValueError):
        tq.quantize_fp8(torch.ones(4, 512), stream=side)
