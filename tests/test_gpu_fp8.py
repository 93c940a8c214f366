"""Block-scaled e4m3: the quantiser bit for bit against its fp32 definition, the
product against the same sum in 64 bits.

Tolerance of a product, derived: a block's 128 products are exact in fp32 and
are added with at most one unit in the last place (2^-23) lost per addition,
128 in all; the scale (one product of two scales) and each block's multiply-add
round once more (2^-24 each, blocks + 2 of them).  All are relative to the sum
of the terms' magnitudes.  A bf16 result adds 2^-8 of its own value."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def up(n, to):
    return -(-n // to) * to


def normal(seed, *shape, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=device)


def ref_quant(x, rows, cols):
    """Codes (uint8, x's shape) and scales [row blocks][column blocks] of fp32 x, from the definition."""
    R, C = x.shape
    f = torch.zeros(up(R, rows), up(C, cols), device=x.device)
    f[:R, :C] = x
    b = f.view(f.shape[0] // rows, rows, f.shape[1] // cols, cols)
    amax = b.abs().amax(dim=(1, 3), keepdim=True)
    s = torch.clamp(amax, min=1e-20) / torch.full_like(amax, 448.0)
    q = torch.clamp(b / s, -448.0, 448.0).to(F8).view(torch.uint8).view(f.shape)[:R, :C]
    return q, s[:, 0, :, 0]


def values(q, s, rows, cols):
    """fp64 values of codes [R][C] under scales [row blocks][column blocks]."""
    sc = s.double().repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(cols, 1)[:, :q.shape[1]]
    return q.contiguous().view(F8).double() * sc


def check_quant(q, s, x, square):
    rq, rs = ref_quant(x, 128 if square else 1, 128)
    C = x.shape[1]
    assert torch.equal(s, rs if square else rs.t())
    raw = q.view(torch.uint8)
    # -0 and 0 are the same value: a quotient that rounds to nothing keeps its sign in both
    assert torch.equal(raw[:, :C], rq)
    assert not raw[:, C:].any()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 4096), (3, 130), (16, 2048), (128, 128), (129, 127), (37, 1410),
                                 (300, 516), (1, 131), (257, 2)])
def test_quantize_forms(cuda_lib, R, C, bf16):
    tq = cuda_lib
    x = normal(R * 7 + C, R, C) * torch.exp(3 * normal(C, R, C))
    if bf16:
        x = x.bfloat16()
    f = x.float()
    check_quant(*tq.quantize_fp8(x), f, False)
    check_quant(*tq.quantize_fp8(x, square=True), f, True)
    for square in (False, True):
        q, s, qt, st = tq.quantize_fp8(x, square=square, transpose=True)
        check_quant(q, s, f, square)
        check_quant(qt, st, f.t().contiguous(), square)
    assert tq.device_status() == 0


def test_quantize_special_values(cuda_lib):
    tq = cuda_lib
    x = normal(5, 6, 256)
    x[0] = 0.0                              # an empty block: the floor's scale, codes 0
    x[1] = torch.finfo(torch.float32).max   # quotients of exactly 448
    x[2] *= 1e-30                           # below the floor
    x[3, :128] = torch.linspace(-1, 1, 128, device="cuda") * 464.0  # past the largest code before scaling
    x[4, 0], x[4, 1:128] = 448.0, torch.arange(1, 128, device="cuda") * 2.0 ** -10  # subnormal codes and their ties
    check_quant(*tq.quantize_fp8(x), x, False)
    check_quant(*tq.quantize_fp8(x, square=True), x, True)
    y = x.clone()
    y[5, 3], y[0, 7] = float("nan"), float("inf")
    q, s = tq.quantize_fp8(y)
    assert torch.isnan(q[5, 3].float()) and torch.isnan(q[0, 7].float())
    assert torch.equal(q[1:5].view(torch.uint8), tq.quantize_fp8(x)[0][1:5].view(torch.uint8))
    assert not torch.isnan(q[5, 4:].float()).any()


@pytest.mark.parametrize("R,C,bf16,gain", [(1, 1, False, True), (5, 4096, False, True), (16, 130, True, False),
                                           (3, 1410, True, True)])
def test_quantize_after_rmsnorm(cuda_lib, R, C, bf16, gain):
    tq = cuda_lib
    x = normal(C, R, C) * 3.0
    if bf16:
        x = x.bfloat16()
    g = 1.0 + 0.2 * normal(9, C) if gain else None
    d = x.double()
    r = 1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / C + torch.tensor(1e-6).double().item())
    f = (d * r * (g.double() if gain else 1.0)).float()
    check_quant(*tq.quantize_fp8(x, rmsnorm=True, rms_gain=g), f, False)


def operands(tq, M, N, K, w_rows, seed=0):
    x, w = normal(seed + 1, M, K), 0.05 * normal(seed + 2, N, K) * torch.exp(normal(seed + 3, N, 1))
    xq, sx = tq.quantize_fp8(x)
    wq, sw = tq.quantize_fp8(w, square=not w_rows)
    xv = values(xq[:, :K], sx.t(), 1, 128)
    wv = values(wq[:, :K], sw.t() if w_rows else sw, 1 if w_rows else 128, 128)
    return xq, sx, wq, sw, xv, wv


def check_product(y, xv, wv, K, plus=None):
    ref, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    if plus is not None:
        ref, mag = ref + plus.double(), mag + plus.double().abs()
    nblk = -(-K // 128)
    tol = mag * (128 * 2.0 ** -23 + (nblk + 3) * 2.0 ** -24)
    if y.dtype == torch.bfloat16:
        tol = tol + ref.abs() * 2.0 ** -8
    err = (y.double() - ref).abs()
    assert torch.isfinite(y.float()).all()
    assert (err <= tol + 1e-30).all(), f"{(err - tol).max().item()} over, at {int((err > tol).sum())} of {err.numel()}"


SHAPES = [(1, 1, 1), (1, 128, 128), (3, 7, 5), (16, 130, 257), (5, 128, 8192), (17, 1000, 1410), (33, 64, 4096),
          (64, 300, 129), (65, 129, 640), (129, 257, 1111), (300, 520, 2000), (1000, 1536, 512), (513, 1024, 300),
          (2048, 4100, 256), (16, 20000, 128)]


@pytest.mark.parametrize("w_rows", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(cuda_lib, M, N, K, w_rows):
    tq = cuda_lib
    xq, sx, wq, sw, xv, wv = operands(tq, M, N, K, w_rows)
    check_product(tq.fp8_gemm(xq, sx, wq, sw, K, w_rows=w_rows), xv, wv, K)
    check_product(tq.fp8_gemm(xq, sx, wq, sw, K, w_rows=w_rows, bf16=True), xv, wv, K)
    y0 = normal(4, M, N)
    y = y0.clone()
    fl = tq.FLAG_ACCUMULATE | tq.FLAG_WEIGHTS_STATIC | (tq.FLAG_FP8_W_ROWS if w_rows else 0)
    tq.fp8_gemm_(xq, sx, wq, sw, K, fl, y)
    check_product(y, xv, wv, K, plus=y0)
    assert tq.device_status() == 0


def test_product_of_unequal_scales(cuda_lib):
    """Every scale its own power of two and every product 1: each output is a sum the test can write down, so a
    scale taken from another block, row or token shows."""
    tq = cuda_lib
    M, N, K = 70, 300, 1000
    kb, nb = -(-K // 128), -(-N // 128)
    one = torch.ones(1, device="cuda").to(F8)
    xq, wq = one.expand(M, up(K, 16)).contiguous(), one.expand(N, up(K, 16)).contiguous()
    sx = 2.0 ** -((torch.arange(kb, device="cuda")[:, None] * 3 + torch.arange(M, device="cuda")[None] * 5) % 7).float()
    sw = 2.0 ** -((torch.arange(nb, device="cuda")[:, None] * 2 + torch.arange(kb, device="cuda")[None] * 3) % 5).float()
    per = torch.full((kb,), 128.0, device="cuda")
    per[-1] = K - 128 * (kb - 1)
    ref = torch.einsum("bm,nb,b->mn", sx, sw.repeat_interleave(128, 0)[:N], per)
    assert torch.equal(tq.fp8_gemm(xq, sx.contiguous(), wq, sw.contiguous(), K), ref)
    swr = 2.0 ** -((torch.arange(kb, device="cuda")[:, None] + torch.arange(N, device="cuda")[None] * 3) % 5).float()
    ref = torch.einsum("bm,bn,b->mn", sx, swr, per)
    assert torch.equal(tq.fp8_gemm(xq, sx.contiguous(), wq, swr.contiguous(), K, w_rows=True), ref)


@pytest.mark.parametrize("M,N,K", [(16, 4096, 4096), (333, 1000, 1410), (1024, 2048, 1024)])
def test_repeatable_and_captured(cuda_lib, M, N, K):
    """The same bits every time, on another stream, and from a replayed graph of quantiser and product."""
    tq = cuda_lib
    x, w = normal(1, M, K), normal(2, N, K)
    wq, sw = tq.quantize_fp8(w, square=True)

    def step(out):
        q, s = tq.quantize_fp8(x)
        tq.fp8_gemm_(q, s, wq, sw, K, 0, out)

    first = torch.empty(M, N, device="cuda")
    step(first)
    for _ in range(3):
        again = torch.empty_like(first)
        step(again)
        assert torch.equal(first, again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(first)
    with torch.cuda.stream(side):
        step(out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, first)
    x.mul_(-1.0)
    for _ in range(3):
        out.zero_()
        g.replay()
    assert torch.equal(out, -first)
    assert tq.device_status() == 0


def test_nothing_outside_is_written(cuda_lib):
    tq = cuda_lib
    M, N, K = 19, 77, 333
    guard = 4096

    def guarded(shape, dt):
        n = int(torch.tensor(shape).prod()) * torch.empty(0, dtype=dt).element_size()
        buf = torch.full((up(n, 16) + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, n, buf[guard:guard + n].view(dt).view(shape)

    x = normal(3, M, K)
    q, s = guarded((M, up(K, 16)), F8), guarded((-(-K // 128), M), torch.float32)
    qt, st = guarded((K, up(M, 16)), F8), guarded((-(-M // 128), K), torch.float32)
    tq.quantize_fp8_(x, 0, q[2], s[2], qt[2], st[2])
    wq, sw = tq.quantize_fp8(normal(4, N, K), square=True)
    y, yb = guarded((M, N), torch.float32), guarded((M, N), torch.bfloat16)
    tq.fp8_gemm_(q[2], s[2], wq, sw, K, 0, y[2])
    tq.fp8_gemm_(q[2], s[2], wq, sw, K, tq.FLAG_BF16_OUTPUT, yb[2])
    torch.cuda.synchronize()
    for buf, n, _ in (q, s, qt, st, y, yb):
        assert (buf[:guard] == 0xA5).all() and (buf[guard + n:] == 0xA5).all()


@pytest.mark.parametrize("M,N,K,bf16", [(40, 50, 60, False), (257, 384, 300, True)])
def test_training_step(cuda_lib, M, N, K, bf16):
    """y, dx, dw of one layer: against the formulas on the quantised operands (the products' tolerance), and
    against differences of the unquantised loss <dy, x w^T> (each factor within 2^-4 of its value: e4m3's half step)."""
    tq = cuda_lib
    x, w, dy = normal(1, M, K), 0.05 * normal(2, N, K), 0.001 * normal(3, M, N)
    if bf16:
        x, dy = x.bfloat16(), dy.bfloat16()
    xq, sx, xt, sxt = tq.quantize_fp8(x, transpose=True)
    dq, sd, dt, sdt = tq.quantize_fp8(dy, transpose=True)
    wq, sw, wt, swt = tq.quantize_fp8(w, square=True, transpose=True)
    y = tq.fp8_gemm(xq, sx, wq, sw, K)
    dx = tq.fp8_gemm(dq, sd, wt, swt, N)
    dw = tq.fp8_gemm(dt, sdt, xt, sxt, M, w_rows=True)
    wv = values(wq[:, :K], sw, 128, 128)
    check_product(y, values(xq[:, :K], sx.t(), 1, 128), wv, K)
    check_product(dx, values(dq[:, :N], sd.t(), 1, 128), wv.t().contiguous(), N)
    check_product(dw, values(dt[:, :M], sdt.t(), 1, 128), values(xt[:, :M], sxt.t(), 1, 128), M)
    X, W, D = x.double(), w.double(), dy.double()

    def loss(X, W):
        return (D * (X @ W.t())).sum()

    for grad, at, mag in ((dx, 0, D.abs() @ W.abs()), (dw, 1, D.abs().t() @ X.abs())):
        u = normal(11 + at, *grad.shape).double()
        h = 1e-3
        step = (loss(X + h * u, W) - loss(X - h * u, W)) if at == 0 else (loss(X, W + h * u) - loss(X, W - h * u))
        # two quantised factors, 2^-4 of each element's value (or, for the smallest, of the block's smallest step)
        bound = (mag * u.abs()).sum() * (2 * 2.0 ** -4 + 2.0 ** -8)
        assert abs((grad.double() * u).sum() - step / (2 * h)) <= bound


@pytest.mark.parametrize("R,C", [(1, 300001), (300001, 1), (2, 131072)])
def test_quantize_long(cuda_lib, R, C):
    tq = cuda_lib
    x = normal(R + C, R, C)
    check_quant(*tq.quantize_fp8(x), x, False)
    q, s, qt, st = tq.quantize_fp8(x, square=True, transpose=True)
    check_quant(q, s, x, True)
    check_quant(qt, st, x.t().contiguous(), True)


@pytest.mark.parametrize("M,N,K", [(2, 40, 300000), (90, 70, 100001)])
def test_product_long(cuda_lib, M, N, K):
    tq = cuda_lib
    for w_rows in (False, True):
        xq, sx, wq, sw, xv, wv = operands(tq, M, N, K, w_rows)
        check_product(tq.fp8_gemm(xq, sx, wq, sw, K, w_rows=w_rows), xv, wv, K)
    assert tq.device_status() == 0


def test_past_32_bit_offsets(cuda_lib):
    """More than 2^31 elements in, and out: the last rows against the same rows alone."""
    tq = cuda_lib
    R, C = 132000, 16400
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    x[:1000] = 0
    x[-300:] = normal(1, 300, C).bfloat16()
    q, s = tq.quantize_fp8(x)
    q2, s2 = tq.quantize_fp8(x[-300:].contiguous())
    assert torch.equal(q[-300:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[:, -300:], s2)
    del x, q, s
    M, N, K = 66000, 33000, 16
    a, b = normal(2, M, K), normal(3, N, K)
    aq, sa = tq.quantize_fp8(a)
    bq, sb = tq.quantize_fp8(b, square=True)
    y = tq.fp8_gemm(aq, sa, bq, sb, K, bf16=True)
    av, bv = values(aq[:, :K], sa.t(), 1, 128), values(bq[:, :K], sb, 128, 128)
    check_product(y[-300:], av[-300:], bv, K)
    check_product(y[:300, -300:], av[:300], bv[-300:], K)
    assert tq.device_status() == 0


def test_quantize_negative_zero(cuda_lib):
    """-0 / s is -0, and so is a negative value over an infinite scale: the sign stays in the code (0x80)."""
    tq = cuda_lib
    x = normal(7, 130, 260)
    x[1::5, ::2] = -0.0
    x[3] = -0.0
    x[:, 9] = -0.0
    x[8, :128] *= -1e-30                    # below the floor: quotients that round to nothing
    check_quant(*tq.quantize_fp8(x), x, False)
    for square in (False, True):
        q, s, qt, st = tq.quantize_fp8(x, square=square, transpose=True)
        check_quant(q, s, x, square)
        check_quant(qt, st, x.t().contiguous(), square)
    assert (tq.quantize_fp8(x)[0].view(torch.uint8)[3, :260] == 0x80).all()
    x[4, 3] = float("inf")
    raw = tq.quantize_fp8(x)[0].view(torch.uint8)[4, :128]
    want = torch.where(torch.signbit(x[4, :128]), 0x80, 0)
    assert torch.equal(torch.cat((raw[:3], raw[4:])).long(), torch.cat((want[:3], want[4:])))
    # RMSNorm of 0 under a negative gain
    z, g = normal(8, 2, 300), normal(9, 300)
    z[:, ::3] = 0.0
    d = z.double()
    f = (d * (1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / 300 + torch.tensor(1e-6).double().item())) * g.double()).float()
    check_quant(*tq.quantize_fp8(z, rmsnorm=True, rms_gain=g), f, False)


@pytest.mark.parametrize("C", [1, 130, 1411])
def test_padding_of_rows_without_a_finite_norm(cuda_lib, C):
    """A row with a NaN, and an empty row with eps 0 (whose factor is infinite): the bytes past cols stay zero."""
    tq = cuda_lib
    x = normal(C, 3, C)
    x[0, C // 2], x[1] = float("nan"), 0.0
    q, _ = tq.quantize_fp8(x, rmsnorm=True, rms_eps=0.0)
    assert not q.view(torch.uint8)[:, C:].any()
    assert torch.isnan(q[:2, :C].float()).all()
    assert torch.equal(q[2:].view(torch.uint8), tq.quantize_fp8(x[2:].clone(), rmsnorm=True, rms_eps=0.0)[0].view(torch.uint8))


def test_quantize_infinite_scale(cuda_lib):
    """An infinity's block has an infinite scale in every form and its finite elements codes of 0 with their signs."""
    tq = cuda_lib
    x = normal(12, 140, 300)
    x[5, 7], x[130, 299] = float("inf"), -float("inf")

    def check(q, s, v, rows):
        R, C = v.shape
        want = torch.zeros(up(R, rows) // rows, up(C, 128) // 128, dtype=torch.bool, device="cuda")
        for r, c in torch.nonzero(torch.isinf(v)).tolist():
            want[r // rows, c // 128] = True
        assert torch.equal(torch.isinf(s), want)
        in_block = want.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :C]
        code = q.view(torch.uint8)[:, :C].long()
        finite = in_block & torch.isfinite(v)
        assert torch.equal(code[finite], torch.where(torch.signbit(v[finite]), 0x80, 0))
        assert torch.isnan(q[:, :C].float()[torch.isinf(v)]).all()
        rq, _ = ref_quant(torch.where(in_block, torch.zeros_like(v), v), rows, 128)
        assert torch.equal(code[~in_block], rq.long()[~in_block])
        assert not q.view(torch.uint8)[:, C:].any()

    q, s = tq.quantize_fp8(x)
    check(q, s.t(), x, 1)
    check(*tq.quantize_fp8(x, square=True), x, 128)
    for square in (False, True):
        q, s, qt, st = tq.quantize_fp8(x, square=square, transpose=True)
        check(q, s if square else s.t(), x, 128 if square else 1)
        check(qt, st if square else st.t(), x.t().contiguous(), 128 if square else 1)
    assert tq.device_status() == 0


@pytest.mark.parametrize("M,N,K,bf16", [(40, 50, 60, False), (257, 384, 300, True), (1000, 640, 1100, False)])
def test_gradients_against_the_formula(cuda_lib, M, N, K, bf16):
    """dx and dw against the exact gradients of <dy, x w^T>, and along the steepest direction against its differences.

    Bound, derived: rounding to e4m3 moves each of a term's two factors by at most 2^-4 of its value (elements with
    subnormal codes by 2^-10 / 448 of their block's largest, which is nothing beside the block's mean square), so an
    independent term's squared error is at most (2 * 2^-8 + 2^-16) of its square.  The operands are independent and of
    mean zero, and so are the errors: the squared 2-norms of gradient and error are their terms' sums, and the error's
    norm is at most sqrt(2) 2^-4 = 0.088 of the gradient's, plus their fluctuation, 1 / sqrt of the 2400 and more elements."""
    tq = cuda_lib
    x, w, dy = normal(21, M, K), 0.05 * normal(22, N, K), 0.001 * normal(23, M, N)
    if bf16:
        x, dy = x.bfloat16(), dy.bfloat16()
    _, _, xt, sxt = tq.quantize_fp8(x, transpose=True)
    dq, sd, dt, sdt = tq.quantize_fp8(dy, transpose=True)
    _, _, wt, swt = tq.quantize_fp8(w, square=True, transpose=True)
    dx = tq.fp8_gemm(dq, sd, wt, swt, N).double().cpu()
    dw = tq.fp8_gemm(dt, sdt, xt, sxt, M, w_rows=True).double().cpu()
    assert tq.device_status() == 0
    X, W, D = x.double().cpu(), w.double().cpu(), dy.double().cpu()

    def loss(X, W):
        return (D * (X @ W.t())).sum()

    bound = 2 ** 0.5 * 2.0 ** -4 * (1 + 2400 ** -0.5)
    for grad, exact, at in ((dx, D @ W, 0), (dw, D.t() @ X, 1)):
        size = exact.norm()

        def off(g):
            return (g - exact).norm() / size

        assert off(grad) <= bound
        # the bound is one: none of these keeps it
        for wrong in (torch.zeros_like(grad), -grad, 1.2 * grad, grad.roll(1, 0), grad.roll(1, 1)):
            assert off(wrong) > bound
        u = exact / size
        d = loss(X + u, W) - loss(X - u, W) if at == 0 else loss(X, W + u) - loss(X, W - u)  # the loss is linear in each
        assert abs((grad * u).sum() - d / 2) <= bound * size and bound * size < 0.1 * d / 2
