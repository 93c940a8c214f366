"""The expert layer and the 8-bit product as a decode step uses them: a mixture-of-experts layer with its residual, the
last RMSNorm fused into the quantiser, the output head; eager, captured and replayed on new tokens, beside a dense
ternary layer of the same network."""
import pytest
import torch

from test_gpu_fp8 import check_product, normal, values
from test_gpu_moe import check_y, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 7, 64])
def test_decode_step(cuda_lib, M):
    tq = cuda_lib
    D, F, E, k, V = 1024, 512, 16, 4, 5003
    x, router, layers = make(M, M, D, F, E, True)
    head_q, head_s = tq.quantize_fp8(0.02 * normal(1, V, D), square=True)
    gain = 1.0 + 0.1 * normal(2, D)
    pk, pg = tq.quantize_ternary_pack(0.02 * normal(3, D, D), per_row=True)
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW | tq.FLAG_NORM_TOPK
    ids, w = torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")
    ws = torch.empty(tq.moe_workspace_bytes(M, D, F, E, k, fl), dtype=torch.uint8, device="cuda")
    bws = torch.empty(tq.fused_workspace_bytes(M, D, fl), dtype=torch.uint8, device="cuda")
    h, y = torch.empty_like(x), torch.empty_like(x)
    res = torch.empty_like(x)
    q = torch.empty((M, D), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((D // 128, M), device="cuda")
    logits = torch.empty((M, V), device="cuda")

    def step():  # a dense ternary layer, the experts, the head
        tq.bitlinear_fused_(x, pk, pg, tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW, h, bws)
        tq.moe_swiglu_(h, router, *layers, fl, y, ids, w, ws)
        torch.add(x, y, out=res)
        tq.quantize_fp8_(res, tq.FLAG_RMSNORM, q, s, rms_gain=gain)
        tq.fp8_gemm_(q, s, head_q, head_s, D, tq.FLAG_WEIGHTS_STATIC, logits)

    def check():
        torch.cuda.synchronize()
        ref, mag, rid, _ = reference(h, router, layers, k, True, True, True, 0)
        assert torch.equal(ids.long(), rid)
        check_y(y, ref, mag, k)
        assert torch.equal(res, x + y)
        check_product(logits, values(q, s.t(), 1, 128), values(head_q[:, :D], head_s, 128, 128), D)
        again = tq.quantize_fp8(res, rmsnorm=True, rms_gain=gain)
        assert torch.equal(again[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(again[1], s)
        assert tq.device_status() == 0

    for _ in range(3):
        step()
    check()
    first = logits.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        step()
    logits.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(logits, first)
    x.copy_(normal(50 + M, M, D))
    for _ in range(3):
        g.replay()
    check()


def test_two_captured_steps_with_their_own_workspaces(cuda_lib):
    """Two graphs of the expert layer replayed on two streams at once: the cooperative launches take turns."""
    tq = cuda_lib
    M, D, F, E, k = 8, 512, 512, 8, 2
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW
    work = []
    for seed in (1, 2):
        x, router, layers = make(seed, M, D, F, E, True)
        out = [torch.empty_like(x), torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda"),
               torch.empty(tq.moe_workspace_bytes(M, D, F, E, k, fl), dtype=torch.uint8, device="cuda")]
        tq.moe_swiglu_(x, router, *layers, fl, *out)
        torch.cuda.synchronize()
        want = out[0].clone()
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(4):
                tq.moe_swiglu_(x, router, *layers, fl, *out)
        work.append((g, st, out, want, x, router, layers))
    for _ in range(10):
        for g, st, *_ in work:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, _, out, want, *_ in work:
        assert torch.equal(out[0], want)
    assert tq.device_status() == 0
