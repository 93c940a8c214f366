"""The mixture-of-experts layer against its definition, evaluated with torch: fp64 sums and fp32 values exactly where
the definition rounds (the logits, the rotated values, the codes' scales, each projection's output).

Tolerances, derived: choices of experts are equal (the logits are fp64 sums rounded once, ties go to the lower index).
A weight is an fp64 quotient rounded to fp32: one unit, 2^-23.  The pairs' outputs are the definition's fp32 values, so
y differs by its weights (2^-23 each) and the roundings of top_k multiply-adds (2^-24 each), relative to the sum of the
terms' magnitudes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def full(v, like):
    return torch.full_like(like, v)


def fwht(x):
    shape, h = x.shape, 1
    while h < 512:
        v = x.reshape(-1, 2, h)
        x = torch.stack((v[:, 0] + v[:, 1], v[:, 0] - v[:, 1]), dim=1)
        h *= 2
    return x.reshape(shape) * torch.tensor(512.0 ** -0.5, device=x.device)


def quant(x, rms):
    if rms:
        d = x.double()
        eps = torch.tensor(1e-6, dtype=torch.float32).double().item()
        x = (d * (1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / x.shape[1] + eps))).float()
    x = fwht(x)
    eta = torch.clamp(x.abs().amax(1, keepdim=True), min=1e-6)
    return torch.clamp(torch.round(x * (full(127.0, eta) / eta)), -127, 127), eta / full(127.0, eta)


DECODE = {0: (-1.0, 0.0, 1.0, 0.0), 1: (0.0, 1.0, 0.0, -1.0), 2: (0.0, 1.0, -1.0, 0.0)}  # by code, per layout


def unpack(p, enc):
    t = torch.tensor(DECODE[enc], device=p.device)
    return torch.stack([t[((p >> (2 * j)) & 3).long()] for j in range(4)], dim=-1).flatten(-2)


def proj(codes, s, layer, e, per_row, enc):
    packed, gamma = layer
    acc = (codes.double() @ unpack(packed[e], enc).double().t()).float()  # whole numbers below 2^24
    return acc * ((gamma[e][None, :] if per_row else gamma[e]) * s)


def reference(x, router, layers, k, per_row, rms, norm, enc, clamp=10.0, ids=None, w=None):
    M, E = x.shape[0], layers[0][0].shape[0]
    if router is not None:
        logits = (x.double() @ router.double().t()).float()
        srt = torch.sort(logits, dim=1, descending=True, stable=True)
        ids = srt.indices[:, :k]
        e = torch.exp(logits.double() - srt.values[:, :1].double())
        w = torch.gather(e, 1, ids)
        w = (w / (w if norm else e).sum(1, keepdim=True)).float()
    xq, sx = quant(x, rms)
    y = torch.zeros(M, x.shape[1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    for e in range(E):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if not len(tok):
            continue
        g = proj(xq[tok], sx[tok], layers[0], e, per_row, enc).double()
        u = proj(xq[tok], sx[tok], layers[1], e, per_row, enc).double()
        a = torch.clamp((g / (1.0 + torch.exp(-g)) * u).float(), -clamp, clamp)
        hq, sh = quant(a, rms)
        o = proj(hq, sh, layers[2], e, per_row, enc).double() * w[tok, slot][:, None].double()
        y.index_add_(0, tok, o)
        mag.index_add_(0, tok, o.abs())
    return y, mag, ids, w


def make(seed, M, D, F, E, per_row, scale=0.016):
    g = gen(seed)
    x = torch.randn(M, D, generator=g, device="cuda") * torch.where(torch.rand(D, generator=g, device="cuda") < 0.01, 10.0, 1.0)
    router = 0.05 * torch.randn(E, D, generator=g, device="cuda")
    layers = []
    for rows, cols in ((F, D), (F, D), (D, F)):
        c = torch.randint(0, 3, (E, rows, cols // 4, 4), generator=g, device="cuda", dtype=torch.uint8)
        p = c[..., 0] | c[..., 1] << 2 | c[..., 2] << 4 | c[..., 3] << 6
        n = (E, rows) if per_row else (E,)
        layers.append((p.contiguous(), scale * (0.5 + torch.rand(n, generator=g, device="cuda"))))
    return x, router, layers


def check_y(y, ref, mag, k):
    err = (y.double() - ref).abs()
    tol = mag * ((k + 4) * 2.0 ** -24) + 1e-30
    assert torch.isfinite(y).all()
    assert (err <= tol).all(), f"worst {(err / (mag + 1e-30)).max().item():.3g} of the terms, {int((err > tol).sum())} outputs"


CASES = [  # M, D, F, E, k, per_row, rms, norm
    (1, 512, 512, 1, 1, False, True, True),
    (1, 512, 1024, 8, 2, False, True, True),
    (3, 1024, 512, 5, 5, True, False, False),
    (7, 2048, 1024, 64, 8, True, True, True),
    (64, 512, 512, 256, 8, False, True, True),
    (33, 1536, 2048, 4, 2, True, True, False),      # several problems per expert and a rest
    (17, 512, 8192, 3, 1, False, True, True),       # the longest rows of the down projection
    (5, 8192, 512, 4, 2, True, True, True),         # and of the others
    (64, 512, 512, 2, 2, True, True, True),         # every token on every expert
    (64, 1024, 1536, 40, 16, False, False, True),   # the most slots
    (2, 4608, 2560, 9, 3, True, True, False),       # teams of 9 and 5 warps
    (64, 512, 1024, 3, 2, False, True, True),       # many pairs per expert: several problems of each
    (33, 4608, 1536, 2, 1, True, True, True),       # ... with the short ring of long rows
    (64, 1024, 7168, 5, 1, True, False, False),
    (40, 8192, 1024, 2, 2, False, True, True),
]


@pytest.mark.parametrize("M,D,F,E,k,per_row,rms,norm", CASES)
def test_layer(cuda_lib, M, D, F, E, k, per_row, rms, norm):
    tq = cuda_lib
    x, router, layers = make(M * 13 + D + E, M, D, F, E, per_row)
    y, ids, w = tq.moe_swiglu(x, router, *layers, k, per_row=per_row, rmsnorm=rms, norm_topk=norm)
    ref, mag, rid, rw = reference(x, router, layers, k, per_row, rms, norm, 0)
    assert tq.device_status() == 0
    assert torch.equal(ids.long(), rid)
    assert ((w - rw).abs() <= rw * 2.0 ** -23).all()
    check_y(y, ref, mag, k)
    # the same choice, given: the same bits
    fl = tq.FLAG_FWHT | (tq.FLAG_RMSNORM if rms else 0) | (tq.GAMMA_PER_ROW if per_row else 0)
    y2 = torch.full_like(x, float("nan"))
    ws = torch.full((tq.moe_workspace_bytes(M, D, F, E, k, fl),), 0xFF, dtype=torch.uint8, device="cuda")
    tq.moe_swiglu_(x, None, *layers, fl, y2, ids, w, ws)
    assert torch.equal(y, y2)


# Up to 16 pairs: each of 16 a problem, one expert with all of them, between, one more.
FEW = [(2, 512, 512, 64, 8), (16, 1024, 512, 1, 1), (16, 1536, 2048, 2, 1), (8, 2048, 1536, 8, 2), (2, 8192, 8192, 8, 8),
       (1, 2048, 1024, 64, 16), (5, 1024, 4608, 3, 3), (1, 512, 8192, 40, 9), (17, 1024, 512, 4, 1)]


@pytest.mark.parametrize("M,D,F,E,k", FEW)
def test_few_pairs(cuda_lib, M, D, F, E, k):
    tq = cuda_lib
    x, router, layers = make(M + D + F + E + k, M, D, F, E, True)
    y, ids, w = tq.moe_swiglu(x, router, *layers, k, per_row=True)
    ref, mag, rid, rw = reference(x, router, layers, k, True, True, True, 0)
    assert tq.device_status() == 0
    assert torch.equal(ids.long(), rid)
    check_y(y, ref, mag, k)
    # every other pair without an expert, then all
    for drop in (slice(1, None, 2), slice(None)):
        ids.view(-1)[drop] = -1
        ref, mag, _, _ = reference(x, None, layers, k, True, True, True, 0, ids=ids.long(), w=w)
        fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW
        y = torch.full_like(x, float("nan"))
        ws = torch.empty(tq.moe_workspace_bytes(M, D, F, E, k, fl), dtype=torch.uint8, device="cuda")
        tq.moe_swiglu_(x, None, *layers, fl, y, ids, w, ws)
        check_y(y, ref, mag, k)


@pytest.mark.parametrize("enc", [1, 2])
@pytest.mark.parametrize("M", [2, 40])
def test_layouts(cuda_lib, M, enc):
    tq = cuda_lib
    D, F, E, k = 512, 1024, 3, 2
    x, router, layers = make(5, M, D, F, E, True)
    g = gen(77)  # all four codes: the layouts give each a meaning
    layers = [(torch.randint(0, 256, p.shape, generator=g, device="cuda", dtype=torch.uint8), s) for p, s in layers]
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW | tq.FLAG_NORM_TOPK | (enc << 7)
    y, ids, w = torch.empty_like(x), torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")
    ws = torch.empty(tq.moe_workspace_bytes(M, D, F, E, k, fl), dtype=torch.uint8, device="cuda")
    tq.moe_swiglu_(x, router, *layers, fl, y, ids, w, ws)
    ref, mag, rid, _ = reference(x, router, layers, k, True, True, True, enc)
    assert torch.equal(ids.long(), rid)
    check_y(y, ref, mag, k)


def test_given_choice_with_unused_and_repeated_slots(cuda_lib):
    """Padded tokens (no slot used) give 0; ids outside the experts add nothing; an expert twice in a token counts
    twice; weights of any sign."""
    tq = cuda_lib
    M, D, F, E, k = 9, 512, 1024, 6, 3
    x, _, layers = make(3, M, D, F, E, False)
    ids = torch.tensor([[0, 1, 2], [-1, -1, -1], [5, 5, 1], [6, 3, -7], [2, -1, 2], [4, 4, 4], [2 ** 31 - 1, -2 ** 31, 0],
                        [-1, 0, -1], [3, 2, 1]], dtype=torch.int32, device="cuda")
    w = torch.randn(M, k, generator=gen(4), device="cuda")
    w[3, 0] = w[1, 1] = float("nan")  # of unused slots: never looked at
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM
    y = torch.full_like(x, float("nan"))
    ws = torch.empty(tq.moe_workspace_bytes(M, D, F, E, k, fl), dtype=torch.uint8, device="cuda")
    ids0, w0 = ids.clone(), w.clone()
    tq.moe_swiglu_(x, None, *layers, fl, y, ids, w, ws)
    ref, mag, _, _ = reference(x, None, layers, k, False, True, True, 0, ids=ids.long(), w=w)
    check_y(y, ref, mag, k)
    assert not y[1].any()
    assert torch.equal(ids, ids0) and torch.equal(w.nan_to_num(9.0), w0.nan_to_num(9.0))
    ids.fill_(-1)  # nothing at all
    tq.moe_swiglu_(x, None, *layers, fl, y, ids, w, ws)
    assert not y.any() and tq.device_status() == 0


def test_ties_and_nan_in_the_router(cuda_lib):
    tq = cuda_lib
    M, D, F, E, k = 3, 512, 512, 40, 4
    x, router, layers = make(8, M, D, F, E, False)
    router[5:12] = router[3]           # equal logits: the lower index first
    router[20] = float("nan")          # never chosen while others are left
    router[0] = 0.0                    # logits 0 and -0
    router[1] = -0.0
    _, ids, w = tq.moe_swiglu(x, router, *layers, k)
    clean = router.clone()
    clean[20] = 0.0
    logits = (x.double() @ clean.double().t()).float()
    logits[:, 20] = -float("inf")
    want = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), want)
    assert torch.isfinite(w).all() and ((w.double().sum(1) - 1).abs() <= k * 2.0 ** -24).all()
    # every logit NaN: still k different experts, nothing outside is touched
    y, ids, w = tq.moe_swiglu(x, torch.full_like(router, float("nan")), *layers, k)
    assert torch.equal(ids.long(), torch.arange(k, device="cuda").expand(M, k))
    assert torch.isnan(w).all() and tq.device_status() == 0


def test_sanitized_input(cuda_lib):
    tq = cuda_lib
    M, D, F, E, k = 4, 512, 512, 8, 2
    x, router, layers = make(9, M, D, F, E, True)
    bad = x.clone()
    bad[0, 3], bad[1, 7], bad[2, 500] = float("nan"), float("inf"), -float("inf")
    good = x.clone()
    good[0, 3], good[1, 7], good[2, 500] = 0.0, 40.0, -40.0
    a = tq.moe_swiglu(bad, router, *layers, k, per_row=True, sanitize=True)
    b = tq.moe_swiglu(good, router, *layers, k, per_row=True)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_repeatable_streams_and_graph(cuda_lib):
    """The same bits each time; two calls at once on two streams, each with its workspace; a captured call replayed."""
    tq = cuda_lib
    M, D, F, E, k = 24, 1024, 512, 16, 4
    sets = [make(s, M, D, F, E, True) for s in (1, 2)]
    want = [tq.moe_swiglu(x, r, *l, k, per_row=True)[0] for x, r, l in sets]
    torch.cuda.synchronize()
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW | tq.FLAG_NORM_TOPK
    streams = [torch.cuda.Stream() for _ in sets]
    outs = []
    for (x, r, l), st in zip(sets, streams):
        with torch.cuda.stream(st):
            outs.append([torch.empty_like(x), torch.empty(M, k, dtype=torch.int32, device="cuda"),
                         torch.empty(M, k, device="cuda"),
                         torch.empty(tq.moe_workspace_bytes(M, D, F, E, k, fl), dtype=torch.uint8, device="cuda")])
    torch.cuda.synchronize()
    for _ in range(20):
        for (x, r, l), o, st in zip(sets, outs, streams):
            tq.moe_swiglu_(x, r, *l, fl, o[0], o[1], o[2], o[3], stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w)
    (x, r, l), o, st = sets[0], outs[0], streams[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        tq.moe_swiglu_(x, r, *l, fl, *o, stream=torch.cuda.current_stream())
    x.copy_(sets[1][0])
    o[0].zero_()
    g.replay()
    torch.cuda.synchronize()
    ref, mag, rid, _ = reference(x, r, l, k, True, True, True, 0)
    assert torch.equal(o[1].long(), rid)
    check_y(o[0], ref, mag, k)
    assert tq.device_status() == 0


def test_nothing_outside_is_written(cuda_lib):
    tq = cuda_lib
    M, D, F, E, k = 5, 512, 1024, 7, 3
    x, router, layers = make(6, M, D, F, E, True)
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW
    bufs = []

    def guarded(shape, dt):
        n = int(torch.tensor(shape).prod()) * torch.empty(0, dtype=dt).element_size()
        raw = torch.full(((n + 15) // 16 * 16 + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        bufs.append((raw, n))
        return raw[4096:4096 + n].view(dt).view(shape)
    out = [guarded((M, D), torch.float32), guarded((M, k), torch.int32), guarded((M, k), torch.float32),
           guarded((tq.moe_workspace_bytes(M, D, F, E, k, fl),), torch.uint8)]
    tq.moe_swiglu_(x, router, *layers, fl, *out)
    torch.cuda.synchronize()
    for raw, n in bufs:
        assert (raw[:4096] == 0x5A).all() and (raw[4096 + n:] == 0x5A).all()


def test_agrees_with_the_dense_block(cuda_lib):
    """One expert, weight 1: the SwiGLU block of the same layers.  SiLU is fp64 here and fp32 there, so single codes
    of the down projection may differ by one: each moves an output by gamma * s."""
    tq = cuda_lib
    M, D, F = 16, 1024, 1024
    x, router, layers = make(12, M, D, F, 1, True)
    y, _, w = tq.moe_swiglu(x, router, *layers, 1, per_row=True)
    assert (w == 1).all()
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW
    dense, act = torch.empty_like(x), torch.empty(M, F, device="cuda")
    ws = torch.empty(tq.swiglu_workspace_bytes(M, D, F, fl), dtype=torch.uint8, device="cuda")
    tq.swiglu_mlp_(x, *[(p[0], g[0]) for p, g in layers], fl, dense, ws, 10.0, act)
    _, s = quant(act, True)
    flips = F // 128  # codes that could move, generously: 127 * 4 ulp of a value near a border, over F of them
    assert ((y - dense).abs() <= flips * layers[2][1] * s * 1.001 + dense.abs() * 1e-5).all()


def test_every_pair_on_one_expert(cuda_lib):
    """The most pairs one expert can get: 64 tokens with all 16 slots on it."""
    tq = cuda_lib
    M, D, F, E, k = 64, 512, 512, 20, 16
    x, _, layers = make(21, M, D, F, E, True)
    ids = torch.full((M, k), 13, dtype=torch.int32, device="cuda")
    w = torch.rand(M, k, generator=gen(2), device="cuda")
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW
    y = torch.empty_like(x)
    ws = torch.empty(tq.moe_workspace_bytes(M, D, F, E, k, fl), dtype=torch.uint8, device="cuda")
    tq.moe_swiglu_(x, None, *layers, fl, y, ids, w, ws)
    ref, mag, _, _ = reference(x, None, layers, k, True, True, True, 0, ids=ids.long(), w=w)
    check_y(y, ref, mag, k)
    assert tq.device_status() == 0


def test_weights_past_32_bit_offsets(cuda_lib):
    """160 experts of 8192 x 8192: 2.7 GB per stacked matrix.  Two experts are filled in, the first and the last."""
    tq = cuda_lib
    M, D, F, E, k = 3, 8192, 8192, 160, 2
    x, _, small = make(31, M, D, F, 2, True)
    layers = []
    for p, s in small:
        big = torch.empty((E,) + tuple(p.shape[1:]), dtype=torch.uint8, device="cuda")
        sb = torch.empty((E, s.shape[1]), device="cuda")
        big[0], big[E - 1], sb[0], sb[E - 1] = p[0], p[1], s[0], s[1]
        layers.append((big, sb))
    ids = torch.tensor([[0, E - 1], [E - 1, 0], [E - 1, E]], dtype=torch.int32, device="cuda")
    w = torch.rand(M, k, generator=gen(3), device="cuda")
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.GAMMA_PER_ROW
    y = torch.empty_like(x)
    ws = torch.empty(tq.moe_workspace_bytes(M, D, F, E, k, fl), dtype=torch.uint8, device="cuda")
    tq.moe_swiglu_(x, None, *layers, fl, y, ids, w, ws)
    near = torch.where(ids == E - 1, 1, torch.where(ids == 0, 0, -1)).long()
    ref, mag, _, _ = reference(x, None, small, k, True, True, True, 0, ids=near, w=w)
    check_y(y, ref, mag, k)
    assert tq.device_status() == 0


@pytest.mark.parametrize("M,D,F,E,k", [(1, 512, 1024, 8, 2), (1, 1536, 6144, 8, 2), (2, 512, 512, 64, 8)])
def test_few_pairs_repeatable_on_two_streams(cuda_lib, M, D, F, E, k):
    """Captured steps of a few pairs, replayed side by side: the same bits every time."""
    tq = cuda_lib
    x, router, layers = make(7 * D + F, M, D, F, E, False)
    want, ids, w = tq.moe_swiglu(x, router, *layers, k)
    fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.FLAG_NORM_TOPK
    runs = []
    for _ in range(2):
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        out = (torch.empty_like(x), torch.empty_like(ids), torch.empty_like(w),
               torch.empty(tq.moe_workspace_bytes(M, D, F, E, k, fl), dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            tq.moe_swiglu_(x, router, *layers, fl, *out)
        runs.append((st, g, out))
    for _ in range(20):
        for st, g, out in runs:
            with torch.cuda.stream(st):
                out[0].fill_(float("nan"))
                for _ in range(5):
                    g.replay()
        torch.cuda.synchronize()
        for _, _, out in runs:
            assert torch.equal(out[0], want) and torch.equal(out[1], ids) and torch.equal(out[2], w)
    assert tq.device_status() == 0


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("M,D,F,E,k", [(1, 512, 1024, 8, 2), (1, 1536, 6144, 8, 2), (4, 1024, 512, 6, 3), (9, 512, 512, 5, 3),
                                       (40, 1024, 1536, 6, 2)])
def test_non_finite_tokens(cuda_lib, M, D, F, E, k, rms):
    """A NaN or an infinity makes its own token's output NaN, as in the definition, and no other's; in a token without
    used slots nobody looks at it."""
    tq = cuda_lib
    x, router, layers = make(M + D, M, D, F, E, True)
    _, ids, w = tq.moe_swiglu(x, router, *layers, k, per_row=True, rmsnorm=rms)
    x[0, D - 5] = float("nan")
    if M > 2:
        x[M - 1, 3] = float("inf")
        x[1], ids[1] = float("nan"), -1
    fl = tq.FLAG_FWHT | tq.GAMMA_PER_ROW | (tq.FLAG_RMSNORM if rms else 0)
    y = torch.empty_like(x)
    ws = torch.empty(tq.moe_workspace_bytes(M, D, F, E, k, fl), dtype=torch.uint8, device="cuda")
    tq.moe_swiglu_(x, None, *layers, fl, y, ids, w, ws)
    ref, mag, _, _ = reference(x, None, layers, k, True, rms, False, 0, ids=ids.long(), w=w)
    bad = [0] if M <= 2 else [0, M - 1]
    assert torch.isnan(ref[bad]).all() and torch.isnan(y[bad]).all()
    rest = [m for m in range(M) if m not in bad]
    if rest:
        check_y(y[rest], ref[rest], mag[rest], k)
        assert not y[1].any()
    # with the router: its logits are NaN, and so are the weights
    y, _, w = tq.moe_swiglu(x, router, *layers, k, per_row=True, rmsnorm=rms)
    assert torch.isnan(y[bad]).all() and torch.isnan(w[bad]).all()
    assert tq.device_status() == 0


@pytest.mark.parametrize("M", [2, 30])
def test_non_finite_scales(cuda_lib, M):
    """A NaN scale of one row of an expert's gate: NaN for the tokens that chose the expert, or, sanitized, a zero."""
    tq = cuda_lib
    D, F, E, k = 512, 1024, 6, 2
    x, router, layers = make(M, M, D, F, E, True)
    want, ids, _ = tq.moe_swiglu(x, router, *layers, k, per_row=True)
    e = int(ids[0, 0])
    layers[0][1][e, 7] = float("nan")
    y, _, _ = tq.moe_swiglu(x, router, *layers, k, per_row=True)
    hit = (ids == e).any(1)
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], want[~hit])
    y, _, _ = tq.moe_swiglu(x, router, *layers, k, per_row=True, sanitize=True)
    layers[0][1][e, 7] = 0.0
    assert torch.equal(y, tq.moe_swiglu(x, router, *layers, k, per_row=True, sanitize=True)[0])
    assert tq.device_status() == 0
