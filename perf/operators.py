"""The mixture-of-experts layer and the block-scaled 8-bit floating-point products: their cases and plain forms.

Two families that stand beside the dense ternary layer of a network:

  moe     a whole mixture-of-experts feed-forward layer for the few tokens of a decode step: a router in full
          precision picks top_k of E experts per token; each expert is the clamped SwiGLU block of three ternary
          layers; the experts' outputs are added with the router's weights.
  quant   quantisation to e4m3 with one fp32 scale per block of 128 (1 x 128 along a row of activations or gradients,
          and, for the products of a training step, along a column with the codes transposed; 128 x 128 for weights).
  linear  what a network keeps out of ternary (the output head, a first or last layer): activations quantised in
          blocks of 128, times weights in e4m3 with a scale per 128 x 128 block.
  train   the same layer in training: y, the input gradient and the weight gradient, each one such product.

`run` computes a case in its plain form, from elementary torch operations, or with `own` by the library's calls.
"""
import math

import torch

own = False

FP8_MAX = 448.0     # largest e4m3 value
FP8_FLOOR = 1e-20   # smallest block maximum that a scale is made of
CLAMP = 10.0        # clamp of the SwiGLU activation
EPS = 1e-6          # RMSNorm epsilon (as an fp32 value, below)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token through a small layer: launch and dependency latency only
        {"name": "moe_1x512x1024_e8k2", "op": "moe", "M": 1, "D": 512, "F": 1024, "E": 8, "k": 2, "per_row": False, "norm": True},
        # one token, the SwiGLU block of the benchmark (1536 -> 6144 -> 1536) as the experts of an 8-expert layer
        {"name": "moe_1x1536x6144_e8k2", "op": "moe", "M": 1, "D": 1536, "F": 6144, "E": 8, "k": 2, "per_row": False, "norm": True},
        # an odd batch over many small experts: most are chosen by one token or none
        {"name": "moe_7x2048x1024_e64k8", "op": "moe", "M": 7, "D": 2048, "F": 1024, "E": 64, "k": 8, "per_row": True, "norm": True},
        # the largest decode batch on few experts: many tokens for each
        {"name": "moe_64x1536x6144_e8k2", "op": "moe", "M": 64, "D": 1536, "F": 6144, "E": 8, "k": 2, "per_row": True, "norm": False},
        # the largest decode batch on many experts: every expert is read, a few tokens each
        {"name": "moe_64x2048x1536_e128k8", "op": "moe", "M": 64, "D": 2048, "F": 1536, "E": 128, "k": 8, "per_row": True, "norm": True},
        # one token through a square 8-bit layer
        {"name": "linear_1x4096x4096", "op": "linear", "M": 1, "N": 4096, "K": 4096, "x_bf16": False, "y_bf16": False, "rms": False},
        # a decode batch through the output head, with the last RMSNorm
        {"name": "linear_16x32000x4096", "op": "linear", "M": 16, "N": 32000, "K": 4096, "x_bf16": False, "y_bf16": False, "rms": True},
        # ragged: no size is a multiple of a tile or a block
        {"name": "linear_333x1000x1410", "op": "linear", "M": 333, "N": 1000, "K": 1410, "x_bf16": True, "y_bf16": True, "rms": False},
        # prefill
        {"name": "linear_2048x11008x4096", "op": "linear", "M": 2048, "N": 11008, "K": 4096, "x_bf16": True, "y_bf16": True, "rms": False},
        # a few rows of activations
        {"name": "quant_9x2048", "op": "quant", "R": 9, "C": 2048, "x_bf16": True, "square": False, "trans": False, "rms": True},
        # a weight matrix of a training step, with its transpose
        {"name": "quant_11008x4096_square", "op": "quant", "R": 11008, "C": 4096, "x_bf16": False, "square": True, "trans": True, "rms": False},
        # a training step of one layer: forward, input gradient, weight gradient
        {"name": "train_2048x5632x2048", "op": "train", "M": 2048, "N": 5632, "K": 2048, "x_bf16": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe", "moe", "linear", "linear", "quant", "train"])
    if op == "moe":
        while True:
            D, F, E = 512 * _log(rng, 1, 16), 512 * _log(rng, 1, 16), _log(rng, 1, 256)
            if E * D * F <= 128 * 2048 * 1536:
                break
        return {"op": op, "M": _log(rng, 1, 64), "D": D, "F": F, "E": E, "k": min(E, _log(rng, 1, 8)),
                "per_row": rng.random() < 0.5, "norm": rng.random() < 0.5}
    if op == "quant":
        while True:
            R, C = _log(rng, 1, 16384), _log(rng, 1, 16384)
            if R * C <= 11008 * 4096:
                break
        square, trans = rng.random() < 0.4, rng.random() < 0.5
        return {"op": op, "R": R, "C": C, "x_bf16": rng.random() < 0.5, "square": square, "trans": trans,
                "rms": not square and not trans and rng.random() < 0.5}  # the norm belongs to activations of a forward pass
    while True:
        M, N, K = _log(rng, 1, 4096), _log(rng, 16, 32000), _log(rng, 16, 8192)
        if M * N * K <= (2048 * 11008 * 4096 if op == "linear" else 2048 * 5632 * 2048):
            break
    c = {"op": op, "M": M, "N": N, "K": K, "x_bf16": rng.random() < 0.5}
    if op == "linear":
        c.update(y_bf16=rng.random() < 0.5, rms=rng.random() < 0.3)
    return c


def _ceil(a, b):
    return -(-a // b)


def work(c):
    if c["op"] == "moe":
        M, D, F, E, k = c["M"], c["D"], c["F"], c["E"], c["k"]
        chosen = E * (1.0 - (1.0 - k / E) ** M)  # experts that some token picks, at an even spread
        gammas = 4 * (2 * F + D if c["per_row"] else 3)
        return {"bytes": 8 * M * D + 4 * E * D + chosen * (3 * D * F / 4 + gammas) + 8 * M * k,
                "flops": 2 * M * E * D + 6 * M * k * D * F}
    if c["op"] == "quant":
        R, C = c["R"], c["C"]
        b = R * C * (3 if c["x_bf16"] else 5)
        s = 4 * _ceil(R, 128) * _ceil(C, 128) if c["square"] else 4 * R * _ceil(C, 128)
        if c["trans"]:
            b += R * C
            s += 4 * _ceil(R, 128) * _ceil(C, 128) if c["square"] else 4 * C * _ceil(R, 128)
        return {"bytes": b + s, "flops": 4 * R * C}
    M, N, K = c["M"], c["N"], c["K"]
    xb = 2 if c["x_bf16"] else 4
    if c["op"] == "linear":
        return {"bytes": M * K * xb + N * K + 4 * _ceil(N, 128) * _ceil(K, 128) + M * N * (2 if c["y_bf16"] else 4),
                "flops": 2 * M * N * K}
    return {"bytes": (M * K + M * N) * xb + 4 * N * K + 4 * (M * N + M * K + N * K), "flops": 6 * M * N * K}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _acts(g, rows, cols, bf16):
    """Activations: normal, with a few channels that are ten times as large, as a network's are."""
    x = _normal(g, rows, cols)
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.004, 10.0, 1.0)
    return x.bfloat16() if bf16 else x


def _packed(g, *shape):
    """Packed ternary codes of normal weights under the absmean rule: 5/16 of them zero, four per byte."""
    v = torch.arange(65536, device="cuda")
    table = torch.zeros(65536, dtype=torch.int64, device="cuda")
    for j in range(4):
        f = (v >> (4 * j)) & 15
        table |= torch.where(f < 5, 1, torch.where(f % 2 == 0, 0, 2)) << (2 * j)
    table = table.to(torch.uint8)
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 25):
        n = min(1 << 25, flat.numel() - a)
        flat[a:a + n] = table[torch.randint(0, 65536, (n,), generator=g, device="cuda")]
    return out


def prepare(c, seed):
    g = _gen(seed)
    s = {"case": dict(c)}
    if c["op"] == "moe":
        M, D, F, E = c["M"], c["D"], c["F"], c["E"]
        s["x"] = _acts(g, M, D, False)
        s["router"] = 0.05 * _normal(g, E, D)
        for name, rows, cols in (("gate", F, D), ("up", F, D), ("down", D, F)):
            n = (E, rows) if c["per_row"] else (E,)
            s[name] = (_packed(g, E, rows, cols // 4), 0.016 * (1.0 + 0.1 * torch.rand(n, generator=g, device="cuda")))
        return s
    if c["op"] == "quant":
        s["x"] = _acts(g, c["R"], c["C"], c["x_bf16"]) * (0.02 if c["square"] else 1.0)
        s["gain"] = 1.0 + 0.1 * _normal(g, c["C"])
        return s
    M, N, K = c["M"], c["N"], c["K"]
    s["x"] = _acts(g, M, K, c["x_bf16"])
    w = 0.02 * _normal(g, N, K)
    if c["op"] == "linear":
        # weights are quantised once, ahead of the calls, and kept in the library's layout: codes in rows of a
        # multiple of 16, one scale per 128 x 128 block
        q, sc = _plain_square(w)
        s["w_q"], s["w_s"] = _pad16(q), sc
        s["gain"] = 1.0 + 0.1 * _normal(g, K)
    else:
        s["w"] = w
        s["dy"] = 0.001 * _acts(g, M, N, c["x_bf16"])
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _pad16(q):
    """e4m3 codes with their rows filled up with zeros to a multiple of 16."""
    out = torch.zeros(q.shape[0], 16 * _ceil(q.shape[1], 16), dtype=torch.uint8, device=q.device)
    out[:, :q.shape[1]] = q.view(torch.uint8)
    return out.view(torch.float8_e4m3fn)


def _fill(x, r, c):
    """x with zero rows and columns up to multiples of r and c."""
    out = torch.zeros(r * _ceil(x.shape[0], r), c * _ceil(x.shape[1], c), dtype=x.dtype, device=x.device)
    out[:x.shape[0], :x.shape[1]] = x
    return out


def _by(a, b):
    """a / b, one of the two a number: an IEEE division (torch turns one by a number into a product)."""
    if isinstance(a, float):
        return torch.full_like(b, a) / b
    return a / torch.full_like(a, b)


def _plain_codes(blocks, dims):
    amax = blocks.abs().amax(dim=dims, keepdim=True)
    scale = _by(torch.clamp(amax, min=FP8_FLOOR), FP8_MAX)
    q = torch.clamp(blocks / scale, -FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return q, scale


def _plain_rows(x):
    """Blocks of 1 x 128: codes as x, scales [blocks of a row][rows]."""
    R, C = x.shape
    f = _fill(x, 1, 128)
    q, s = _plain_codes(f.view(R, -1, 128), 2)
    return q.view(torch.uint8).view(R, -1)[:, :C].contiguous().view(torch.float8_e4m3fn), s[:, :, 0].t().contiguous()


def _plain_square(x):
    """Blocks of 128 x 128: codes as x, scales [row blocks][column blocks]."""
    R, C = x.shape
    f = _fill(x, 128, 128)
    q, s = _plain_codes(f.view(f.shape[0] // 128, 128, f.shape[1] // 128, 128), (1, 3))
    return q.view(torch.uint8).view(f.shape)[:R, :C].contiguous().view(torch.float8_e4m3fn), s[:, 0, :, 0].contiguous()


def _plain_norm(x, gain):
    """RMSNorm in 64 bits, rounded once: what a quantiser rounds next must not depend on the order of a sum."""
    x = x.double()
    eps = torch.tensor(EPS, dtype=torch.float32).double().item()
    r = 1.0 / torch.sqrt((x * x).sum(dim=1, keepdim=True) / x.shape[1] + eps)
    return (x * r * (1.0 if gain is None else gain.double())).float()


def _values(q, s):
    """fp32 values of codes with 1 x 128 scales [blocks][rows]."""
    return q.float() * s.t().repeat_interleave(128, dim=1)[:, :q.shape[1]]


def _values_square(q, s):
    return q.float() * s.repeat_interleave(128, dim=0)[:q.shape[0]].repeat_interleave(128, dim=1)[:, :q.shape[1]]


def _plain_fwht(x):
    """Blockwise 512-point Walsh-Hadamard transform: stages of (a + b, a - b) in 32 bits."""
    shape, h = x.shape, 1
    while h < 512:
        v = x.reshape(-1, 2, h)
        x = torch.stack((v[:, 0] + v[:, 1], v[:, 0] - v[:, 1]), dim=1)
        h *= 2
    return x.reshape(shape) * torch.tensor(512.0 ** -0.5, dtype=torch.float32, device=x.device)


def _plain_int8(x):
    """A token's int8 codes (as fp32 whole numbers) and scale, after RMSNorm and the transform."""
    x = _plain_fwht(_plain_norm(x, None))
    eta = torch.clamp(x.abs().amax(dim=1, keepdim=True), min=1e-6)
    codes = torch.clamp(torch.round(x * _by(127.0, eta)), -127, 127)
    return codes, _by(eta, 127.0)


def _plain_unpack(packed, ids):
    """Ternary values of the experts `ids`, fp32."""
    p = packed[ids]
    return torch.stack([((p >> (2 * j)) & 3) for j in range(4)], dim=-1).flatten(-2).float() - 1.0


def _plain_moe(s):
    c, x = s["case"], s["x"]
    M, k = c["M"], c["k"]
    # the choice of experts stands on comparisons of sums: in 64 bits, rounded once
    logits = (x.double() @ s["router"].double().t()).float()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = order.indices[:, :k]
    e = torch.exp(logits.double() - order.values[:, :1].double())
    w = torch.gather(e, 1, ids)
    w = (w / (w.sum(dim=1, keepdim=True) if c["norm"] else e.sum(dim=1, keepdim=True))).float()
    some = torch.unique(ids)                              # experts that some token picks, U
    xq, sx = _plain_int8(x)

    def product(codes, scale, name, rows):                # [U or 1, M, in] -> [U, M, rows]
        packed, gamma = s[name]
        acc = torch.matmul(codes, _plain_unpack(packed, some).transpose(1, 2))  # whole numbers below 2^24: exact
        return acc * (gamma[some].reshape(len(some), 1, rows if c["per_row"] else 1) * scale)

    gate = product(xq[None], sx[None], "gate", c["F"])
    up = product(xq[None], sx[None], "up", c["F"]).double()
    g = gate.double()
    # 64 bits up to the rounding that the next quantiser starts from
    act = torch.clamp((g / (1.0 + torch.exp(-g)) * up).float(), -CLAMP, CLAMP)
    hq, sh = _plain_int8(act.reshape(-1, c["F"]))
    out = product(hq.reshape(len(some), M, -1), sh.reshape(len(some), M, 1), "down", c["D"])
    at = torch.searchsorted(some, ids)                    # [M, k]
    y = (out[at, torch.arange(M, device=x.device)[:, None]] * w[:, :, None]).sum(dim=1)
    return {"y": y, "ids": ids.int(), "weights": w}


def _plain(s):
    c = s["case"]
    if c["op"] == "moe":
        return _plain_moe(s)
    x = s["x"]
    if c["op"] == "quant":
        f = _plain_norm(x, s["gain"]) if c["rms"] else x.float()
        q, sc = _plain_square(f) if c["square"] else _plain_rows(f)
        out = {"q": q, "s": sc}
        if c["trans"]:
            out["qt"], out["st"] = _plain_square(f.t().contiguous()) if c["square"] else _plain_rows(f.t().contiguous())
        return out
    if c["op"] == "linear":
        f = _plain_norm(x, s["gain"]) if c["rms"] else x.float()
        y = _values(*_plain_rows(f)) @ _values_square(s["w_q"][:, :c["K"]], s["w_s"]).t()
        return {"y": y.bfloat16() if c["y_bf16"] else y}
    f, d = x.float(), s["dy"].float()
    w = _values_square(*_plain_square(s["w"]))
    return {"y": _values(*_plain_rows(f)) @ w.t(),
            "dx": _values(*_plain_rows(d)) @ w,
            "dw": _values(*_plain_rows(d.t().contiguous())) @ _values(*_plain_rows(f.t().contiguous())).t()}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import ternary_bit_linear_b200 as tq

    c, x = s["case"], s["x"]
    if c["op"] == "moe":
        fl = tq.FLAG_FWHT | tq.FLAG_RMSNORM | tq.FLAG_WEIGHTS_STATIC
        fl |= (tq.GAMMA_PER_ROW if c["per_row"] else 0) | (tq.FLAG_NORM_TOPK if c["norm"] else 0)
        if "y" not in s:  # outputs and scratch, kept as a decode loop keeps them
            s["y"] = torch.empty_like(x)
            s["ids"] = torch.empty((c["M"], c["k"]), dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty((c["M"], c["k"]), device="cuda")
            s["ws"] = torch.empty(tq.moe_workspace_bytes(c["M"], c["D"], c["F"], c["E"], c["k"], fl), dtype=torch.uint8, device="cuda")
        tq.moe_swiglu_(x, s["router"], s["gate"], s["up"], s["down"], fl, s["y"], s["ids"], s["weights"], s["ws"], clamp_val=CLAMP)
        return {"y": s["y"], "ids": s["ids"], "weights": s["weights"]}
    if c["op"] == "quant":
        r = tq.quantize_fp8(x, square=c["square"], transpose=c["trans"], rmsnorm=c["rms"], rms_gain=s["gain"] if c["rms"] else None)
        out = {"q": r[0][:, :c["C"]], "s": r[1]}
        if c["trans"]:
            out.update(qt=r[2][:, :c["R"]], st=r[3])
        return out
    if c["op"] == "linear":
        q, sc = tq.quantize_fp8(x, rmsnorm=c["rms"], rms_gain=s["gain"] if c["rms"] else None)
        return {"y": tq.fp8_gemm(q, sc, s["w_q"], s["w_s"], c["K"], bf16=c["y_bf16"])}
    xq, xs, xt, xts = tq.quantize_fp8(x, transpose=True)
    dq, ds, dt, dts = tq.quantize_fp8(s["dy"], transpose=True)
    wq, wsc, wt, wts = tq.quantize_fp8(s["w"], square=True, transpose=True)
    return {"y": tq.fp8_gemm(xq, xs, wq, wsc, c["K"]),
            "dx": tq.fp8_gemm(dq, ds, wt, wts, c["N"]),
            "dw": tq.fp8_gemm(dt, dts, xt, xts, c["M"], w_rows=True)}


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.  Where the definition itself rounds (the fp32 values that a quantiser sees, a scale, a
# code), the rounding is made explicitly; everything else is unrounded.
# ---------------------------------------------------------------------------
def _r32(v):
    return v.float().double()


def _e4m3(t):
    """Nearest e4m3 value, ties to even mantissas: 3 bits after the leading one, exponents from -6."""
    e = torch.floor(torch.log2(torch.clamp(t.abs(), min=2.0 ** -20)))
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3.0)
    return torch.clamp(torch.round(t / step) * step, -FP8_MAX, FP8_MAX)


def _exact_blocks(v, rows, cols):
    """Per block of rows x cols of v (fp32 values in 64 bits): code values and, spread over v's shape, the scales."""
    R, C = v.shape
    br, bc = torch.arange(R, device=v.device) // rows, torch.arange(C, device=v.device) // cols
    block = br[:, None] * _ceil(C, cols) + bc[None, :]
    amax = torch.zeros(_ceil(R, rows) * _ceil(C, cols), dtype=torch.float64, device=v.device)
    amax.scatter_reduce_(0, block.reshape(-1), v.abs().reshape(-1), "amax")
    scale = _r32(torch.clamp(amax, min=torch.tensor(FP8_FLOOR, dtype=torch.float32).double().item()) / FP8_MAX)
    spread = scale[block]
    return _e4m3(_r32(v / spread)), spread, scale.view(_ceil(R, rows), _ceil(C, cols))


def _exact_norm(x, gain):
    x = x.double()
    mean = x.pow(2).mean(dim=1, keepdim=True) + torch.tensor(EPS, dtype=torch.float32).double().item()
    y = x * mean.pow(-0.5)
    return _r32(y if gain is None else y * gain.double())


def _exact_int8(x):
    """The definition's int8 codes: the transform as nine sums and differences of fp32 values over the bits of a
    position, each rounded to fp32."""
    v = _exact_norm(x, None)
    v = v.view(-1, *[2] * 9)
    for bit in range(9, 0, -1):  # the lowest bit of the position is the last axis
        a, b = v.select(bit, 0), v.select(bit, 1)
        v = _r32(torch.stack((a + b, a - b), dim=bit))
    v = _r32(v.reshape(x.shape) * torch.tensor(512.0 ** -0.5, dtype=torch.float32).double().item())
    eta = torch.clamp(v.abs().amax(dim=1, keepdim=True), min=torch.tensor(1e-6, dtype=torch.float32).double().item())
    codes = torch.clamp(torch.round(_r32(v * _r32(127.0 / eta))), -127, 127)
    return codes, _r32(eta / 127.0)


def _exact_moe(s):
    c, x = s["case"], s["x"]
    M, k, D, F = c["M"], c["k"], c["D"], c["F"]
    logits = _r32(torch.einsum("md,ed->me", x.double(), s["router"].double()))
    # the k largest, ties to the lower index: by rank, counted
    above = (logits[:, None, :] > logits[:, :, None]).sum(dim=2)
    index = torch.arange(c["E"], device=x.device)
    above += ((logits[:, None, :] == logits[:, :, None]) & (index[None, None, :] < index[None, :, None])).sum(dim=2)
    ids = torch.argsort(above, dim=1)[:, :k]
    p = torch.softmax(logits, dim=1)
    w = torch.gather(p, 1, ids)
    if c["norm"]:
        w = w / w.sum(dim=1, keepdim=True)
    shifts = torch.tensor([0, 2, 4, 6], device=x.device, dtype=torch.uint8)

    def layer(codes, scale, name, e, rows, cols):  # one expert's ternary layer on the tokens given
        packed, gamma = s[name]
        t = ((packed[e].reshape(rows, cols // 4, 1) >> shifts) & 3).reshape(rows, cols).double() - 1.0
        return _r32(codes @ t.t()) * _r32(gamma[e].double().reshape(1, -1) * scale)

    xq, sx = _exact_int8(x)
    y = torch.zeros(M, D, dtype=torch.float64, device=x.device)
    for e in torch.unique(ids).tolist():
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        g = _r32(layer(xq[tok], sx[tok], "gate", e, F, D))
        u = _r32(layer(xq[tok], sx[tok], "up", e, F, D))
        a = torch.clamp(_r32(g * torch.sigmoid(g) * u), -CLAMP, CLAMP)
        hq, sh = _exact_int8(a)
        y.index_add_(0, tok, layer(hq, sh, "down", e, D, F) * w[tok, slot][:, None])
    return {"y": y, "ids": None, "weights": w}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "moe":
        return _exact_moe(s)
    x = s["x"]
    if c["op"] in ("quant", "linear"):
        v = _exact_norm(x, s["gain"]) if c["rms"] else x.double()
        if c["op"] == "quant":
            side = (128, 128) if c["square"] else (1, 128)
            q, _, sc = _exact_blocks(v, *side)
            out = {"q": q, "s": sc if c["square"] else sc.t()}
            if c["trans"]:
                q, _, sc = _exact_blocks(v.t().contiguous(), *side)
                out.update(qt=q, st=sc if c["square"] else sc.t())
            return out
        q, sc, _ = _exact_blocks(v, 1, 128)
        n, kk = torch.arange(c["N"], device=x.device) // 128, torch.arange(c["K"], device=x.device) // 128
        w = s["w_q"][:, :c["K"]].double() * s["w_s"].double()[n[:, None], kk[None, :]]
        return {"y": torch.einsum("mk,nk->mn", q * sc, w)}
    times = lambda t: t[0] * t[1]  # noqa: E731
    v, d = x.double(), s["dy"].double()
    w = times(_exact_blocks(s["w"].double(), 128, 128))
    return {"y": times(_exact_blocks(v, 1, 128)) @ w.t(), "dx": times(_exact_blocks(d, 1, 128)) @ w,
            "dw": times(_exact_blocks(d, 128, 1)).t() @ times(_exact_blocks(v, 128, 1))}
