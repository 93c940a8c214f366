"""The allocating calls on a stream that is given: the stream is kept busy, so that whatever they allocate and drop is
still wanted when the current stream allocates and writes next."""
import pytest
import torch

from test_gpu_fp8 import normal
from test_gpu_moe import make

pytestmark = pytest.mark.gpu

BUSY = 40_000_000  # clock cycles, some 20 ms


def calls(tq):
    """(call on a stream, bytes of the buffers it takes)"""
    M, D, F, E, k = 24, 1024, 512, 16, 4
    x, router, layers = make(1, M, D, F, E, True)
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW
    yield "moe", lambda s: tq.moe_swiglu(x, router, *layers, k, per_row=True, stream=s), [
        tq.moe_workspace_bytes(M, D, F, E, k, fl), 4 * M * D]
    a = normal(2, 300, 1000)
    yield "quantize", lambda s: tq.quantize_fp8(a, transpose=True, stream=s), [300 * 1008, 1000 * 304]
    xq, sx = tq.quantize_fp8(a)
    wq, sw = tq.quantize_fp8(normal(3, 500, 1000), square=True)
    yield "product", lambda s: tq.fp8_gemm(xq, sx, wq, sw, 1000, stream=s), [300 * 500 * 4]
    p, g = tq.quantize_ternary_pack(normal(4, 512, 1024), True)
    yield "fused", lambda s: tq.bitlinear_fused(x, p, g, True, stream=s), [tq.fused_workspace_bytes(M, D, fl), 4 * M * 512]
    w = normal(5, 512, 4096)
    yield "pack", lambda s: tq.quantize_ternary_pack(w, False, stream=s), [tq.pack_workspace_bytes(512, 4096, 0), 512 * 1024]


def as_bytes(out):
    return [t.view(torch.uint8).clone() for t in (out if isinstance(out, tuple) else (out,))]


def same(out, want):
    return all(torch.equal(a, b) for a, b in zip(as_bytes(out), want, strict=True))


def test_scratch_outlives_the_call(cuda_lib):
    tq = cuda_lib
    for name, call, sizes in calls(tq):
        want = as_bytes(call(None))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for _ in range(3):
            with torch.cuda.stream(side):
                torch.cuda._sleep(BUSY)
            out = call(side)
            junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4) if n]
            torch.cuda.current_stream().synchronize()
            side.synchronize()
            assert same(out, want), name
            del junk, out
    assert tq.device_status() == 0


def test_results_outlive_their_readers(cuda_lib):
    """A result dropped while the current stream has still to read it: the next call on the side stream, of the same
    sizes, takes other memory."""
    tq = cuda_lib
    for name, call, _ in calls(tq):
        want = as_bytes(call(None))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        out = call(side)
        side.synchronize()
        torch.cuda._sleep(BUSY)
        kept = as_bytes(out)  # reads that wait behind the sleep
        del out
        with torch.cuda.stream(side):
            for _ in range(3):
                for t in kept:
                    torch.full_like(t, 0xFF)
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want, strict=True)), name
    assert tq.device_status() == 0


def test_captured_on_the_given_stream(cuda_lib):
    tq = cuda_lib
    for name, call, _ in calls(tq):
        want = as_bytes(call(None))
        torch.cuda.synchronize()
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=st):
            out = call(torch.cuda.current_stream())
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert same(out, want), name
    assert tq.device_status() == 0


def test_captured_on_a_second_stream(cuda_lib):
    """A branch of a graph: the call on another stream than the captured one, joined again, its results read there."""
    tq = cuda_lib
    for name, call, _ in calls(tq):
        want = as_bytes(call(None))
        torch.cuda.synchronize()
        g, st, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=st):
            side.wait_stream(st)
            out = call(side)
            st.wait_stream(side)
            read = as_bytes(out)
            del out
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(read, want, strict=True)), name
    assert tq.device_status() == 0
