"""The root-mean-square norm around an MoE layer and the layer's products in microscaled 4-bit floating point, as a
user of the library calls them: what is run, on which inputs, and what each pass cannot do without.

A case names its operator in ``op``:

* ``norm``   h = x + r, y = h / rms(h) * w (moe_rms_norm); without a residual r: h = x
* ``norm8``  the same, y leaving in 8-bit integers for a product with 8-bit weights (moe_rms_norm_i8, moe_matmul_i8)
* ``grad``   the norm's gradients for h and for w, with the gradient that reaches h past the norm added
             (moe_rms_norm_grad)
* ``mx4``    rows quantized on the fly, then the grouped product with 4-bit weights (moe_quantize_mx4, moe_matmul_mx4)
* ``round4`` a matrix to 4 bits and back: the values that the codes stand for (moe_quantize_mx4, moe_dequantize_mx4)

Microscaled 4 bits: 32 consecutive values share a scale 2^(s - 127), s = max(0, floor(log2 max|v|) - 2 + 127) in 8
bits; each is one of +-{0, 1/2, 1, 3/2, 2, 3, 4, 6} times it, the nearest one (ties to the even code, beyond 6 to 6).
Codes lie two to a byte, the earlier value in the low half; a row's scales are padded to a multiple of 16.

Sizes: ``rows`` rows of ``K`` values; products with weights of ``N`` rows, ``G`` groups of them (``0``: one group, no
offsets), gathered from ``tokens`` > 0 token rows.  ``spread`` says how the rows fall on the groups: ``even`` (a
balanced router), ``skew`` (popularity 1/rank^1.1, several groups empty), ``one``.

Where ``own`` is false the same values come from elementary torch operations in float32.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
MOST_BYTES = 3e9     # a drawn case's operands and results
MOST_FLOPS = 1.2e12  # a drawn case's product


def listed():
    return [
        # decoding one token of the 7168-wide model: latency counts
        dict(name="norm_one", op="norm", dtype="bf16", w="bf16", rows=1, K=7168, residual=True),
        # a prompt of 8192 tokens
        dict(name="norm_prefill", op="norm", dtype="bf16", w="bf16", rows=8192, K=7168, residual=True),
        # decoding 64 tokens: the norm before an expert's gate that is stored in 8 bits
        dict(name="norm8_decode", op="norm8", dtype="bf16", w="bf16", rows=64, K=7168, N=2048, residual=True),
        # the same expert on a prompt of 8192 tokens
        dict(name="norm8_prefill", op="norm8", dtype="bf16", w="bf16", rows=8192, K=7168, N=2048, residual=True),
        # training on 16384 tokens, the residual stream's gradient added, the weight kept in float32
        dict(name="grad_train", op="grad", dtype="bf16", w="f32", rows=16384, K=7168, residual=True),
        # a small fp32 model of odd width
        dict(name="grad_odd_f32", op="grad", dtype="f32", w="f32", rows=777, K=1001, residual=False),
        # the dense first layer's gate at decode: 64 rows, one group, the weights streamed as half bytes
        dict(name="mx4_decode", op="mx4", dtype="bf16", G=0, rows=64, N=18432, K=7168, tokens=0, spread="one"),
        # decoding 64 tokens, top-8 of 384 experts: the down product, about one row an expert
        dict(name="mx4_experts", op="mx4", dtype="bf16", G=384, rows=512, N=7168, K=2048, tokens=0, spread="even"),
        # the dense layer's gate on a prompt of 8192 tokens
        dict(name="mx4_prefill", op="mx4", dtype="bf16", G=0, rows=8192, N=18432, K=7168, tokens=0, spread="one"),
        # an eighth of the experts on one GPU: rows gathered from 1024 tokens, unevenly, some experts empty
        dict(name="mx4_skew", op="mx4", dtype="bf16", G=48, rows=8192, N=2048, K=7168, tokens=1024, spread="skew"),
        # the tiny fp32 layer's expert weights of the tests and the benchmark: latency counts
        dict(name="round4_tiny_f32", op="round4", dtype="f32", rows=16 * 128, K=256),
        # the dense layer's gate weight on its way to 4 bits
        dict(name="round4_dense", op="round4", dtype="bf16", rows=18432, K=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A row's length: most often a multiple of 64 as models have them, sometimes of 8, sometimes anything."""
    v = _log(rng, lo, hi)
    step = rng.choice((64, 64, 64, 8, 1))
    return max(step, v // step * step)


def draw(rng):
    while True:
        op = rng.choice(("norm", "norm", "norm8", "grad", "grad", "mx4", "mx4", "mx4", "round4"))
        dtype = "f32" if rng.random() < 0.25 else "bf16"
        if op in ("norm", "norm8", "grad"):
            case = dict(op=op, dtype=dtype, w=rng.choice(("bf16", "f32")), rows=_log(rng, 1, 32768),
                        K=_size(rng, 64, 18432), residual=rng.random() < 0.6)
            if op == "norm8":
                case["N"] = _size(rng, 64, 4096)
        elif op == "round4":
            case = dict(op=op, dtype=dtype, rows=_log(rng, 1, 65536), K=32 * _log(rng, 2, 576))
        else:
            G = rng.choice((0, _log(rng, 1, 384)))
            case = dict(op=op, dtype=dtype, G=G, rows=_log(rng, 1, 32768), N=_size(rng, 64, 18432 if G < 4 else 7168),
                        K=32 * _log(rng, 2, 224), tokens=0, spread="one" if G == 0 else rng.choice(("even", "even", "skew")))
            if rng.random() < 0.3:
                case["tokens"] = max(1, case["rows"] // rng.choice((2, 4, 8)))
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return case


def _popularity(case):
    G = max(1, case["G"])
    p = 1.0 / np.arange(1, G + 1) ** 1.1 if case["spread"] == "skew" else np.ones(G)
    return p / p.sum()


def _scale_cols(K):
    return (K + 511) // 512 * 16


def _mx4_weight(gen, G, N, K):
    """Weights already stored in 4 bits: the codes that normally distributed values get, and scales to match."""
    v = torch.randn(1 << 17, generator=gen, device="cuda") * 2.2
    c = _codes4(v.clamp(-7.9, 7.9)).view(-1, 2)
    pairs = (c[:, 0] | c[:, 1] << 4).to(torch.uint8)
    codes = torch.empty((G, N, K // 2), dtype=torch.uint8, device="cuda")
    for g in range(G):
        codes[g] = pairs[torch.randint(0, 1 << 16, (N, K // 2), generator=gen, device="cuda", dtype=torch.int32)]
    unit = 127 + round(math.log2(1.0 / (2.2 * math.sqrt(K))))
    scales = torch.zeros((G, N, _scale_cols(K)), dtype=torch.uint8, device="cuda")
    scales[..., :K // 32] = torch.randint(unit - 1, unit + 2, (G, N, K // 32), generator=gen, device="cuda",
                                          dtype=torch.uint8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, rows, K, op = DTYPES[case["dtype"]], case["rows"], case["K"], case["op"]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)

    def activations(n):  # a few large channels
        x = normal(n, K)
        x[:, torch.randperm(K, generator=gen, device="cuda")[:max(1, K // 100)]] *= 6.0
        return x

    s = dict(op=op)
    if op in ("norm", "norm8", "grad"):
        wdt = DTYPES[case["w"]]
        s["weight"] = (normal(K, dtype=torch.float32) * 0.1 + 1.0).to(wdt)
        if op == "grad":
            s["h"], s["dy"] = activations(rows), normal(rows, K) * 0.01
            s["dh"] = normal(rows, K) * 0.01 if case["residual"] else None
            return s
        s["x"], s["r"] = normal(rows, K), activations(rows) if case["residual"] else None
        if op == "norm8":
            s["wq"] = torch.randint(-127, 128, (1, case["N"], K), generator=gen, device="cuda", dtype=torch.int8)
            s["ws"] = (torch.rand((1, case["N"]), generator=gen, device="cuda") * 0.5 + 0.75) / (73.0 * math.sqrt(K))
        return s
    if op == "round4":
        s["x"] = normal(rows, K) * (1.0 / math.sqrt(K))
        return s
    G = max(1, case["G"])
    s["x"] = activations(case["tokens"] or rows)
    s["group_offsets"] = s["row_index"] = None
    rng = np.random.default_rng([int(seed), 1])
    p = _popularity(case)
    ends = np.concatenate([[0], np.cumsum(rng.multinomial(rows, rng.permutation(p) if case["spread"] == "skew" else p))])
    s["ends"] = ends.tolist()
    if case["G"]:
        s["group_offsets"] = torch.from_numpy(ends.astype(np.int32)).cuda()
    if case["tokens"]:
        s["row_index"] = torch.randint(0, case["tokens"], (rows,), generator=gen, device="cuda", dtype=torch.int32)
    s["wq"], s["ws"] = _mx4_weight(gen, G, case["N"], K)
    return s


# ----------------------------------------------------------------- the library's operators
def _own(s):
    import moe_layer_forward_amd as moe

    op = s["op"]
    if op == "norm":
        return moe.moe_rms_norm(s["x"], s["weight"], residual=s["r"], eps=EPS)
    if op == "norm8":
        q, sq, *h = moe.moe_rms_norm_i8(s["x"], s["weight"], residual=s["r"], eps=EPS)
        y_dtype = moe.MOE_BF16 if s["x"].dtype == torch.bfloat16 else moe.MOE_F32
        return (moe.moe_matmul_i8(q, sq, s["wq"], s["ws"], y_dtype=y_dtype), *h)
    if op == "grad":
        return moe.moe_rms_norm_grad(s["dy"], s["h"], s["weight"], dh=s["dh"], eps=EPS)
    q, sq = moe.moe_quantize_mx4(s["x"])
    dtype = moe.MOE_BF16 if s["x"].dtype == torch.bfloat16 else moe.MOE_F32
    if op == "round4":
        return moe.moe_dequantize_mx4(q, sq, dtype)
    return moe.moe_matmul_mx4(q, sq, s["wq"], s["ws"], s["group_offsets"], row_index=s["row_index"], y_dtype=dtype)


# ----------------------------------------------------------------- the plain forms
def _codes4(v):
    """The nearest 4-bit value's code, for values in units of their scale."""
    m = v.abs()
    c = ((m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)).int()
    return c + 8 * (v < 0).int()


def _values4(c):
    """What the codes 0 .. 15 stand for."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=c.device)
    return torch.cat([table, -table])[c.int()]


def _power(e):
    """2^e in float32, exactly (exp2 is not on every device), for the exponents of normal numbers."""
    return ((e.int().clamp(min=-126) + 127) << 23).view(torch.float32)


def _quantized4(x):
    """(codes [rows, K], scales [rows, K / 32, 1] as numbers), both float32 operations."""
    b = x.view(x.shape[0], -1, 32)
    e = torch.frexp(b.abs().amax(dim=2, keepdim=True))[1]  # the maximum is in [2^(e - 1), 2^e)
    scale = _power(e - 3)
    return _codes4(b / scale), scale


def _dequantized4(codes, scales):
    """float32 values of packed codes [.., K / 2] and scales [.., padded]."""
    K = codes.shape[-1] * 2
    c = torch.stack([codes & 15, codes >> 4], dim=-1).view(*codes.shape[:-1], K // 32, 32)
    unit = _power(scales[..., :K // 32].int() - 127)
    return (_values4(c) * unit[..., None]).view(*codes.shape[:-1], K)


def _plain(s):
    op = s["op"]
    if op == "grad":
        h, dy, w = s["h"].float(), s["dy"].float(), s["weight"].float()
        rstd = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
        g = dy * w
        dx = rstd * (g - h * (rstd * rstd * (g * h).mean(dim=1, keepdim=True)))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        dw = (dy * h * rstd).sum(dim=0)
        return dx.to(s["h"].dtype), dw.to(s["weight"].dtype)
    if op in ("norm", "norm8"):
        h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
        f = h.float()
        y = f * (1.0 / torch.sqrt((f * f).mean(dim=1, keepdim=True) + EPS)) * s["weight"].float()
        if op == "norm8":
            a = y.abs().amax(dim=1, keepdim=True)
            q = torch.where(a > 0, torch.round(y * 127.0 / a), torch.zeros_like(y))
            y = (q @ s["wq"][0].float().t()) * (a / 127.0) * s["ws"][0]
        y = y.to(s["x"].dtype)
        return y if op == "norm" and s["r"] is None else (y,) if s["r"] is None else (y, h)
    x = s["x"].float()
    codes, scale = _quantized4(x)
    x = (_values4(codes) * scale).view(x.shape)
    if op == "round4":
        return x.to(s["x"].dtype)
    if s["row_index"] is not None:
        x = x[s["row_index"].long()]
    y = torch.empty((x.shape[0], s["wq"].shape[1]), dtype=s["x"].dtype, device=x.device)
    for g, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])):
        if a < b:
            y[a:b] = (x[a:b] @ _dequantized4(s["wq"][g], s["ws"][g]).t()).to(y.dtype)
    return y


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------- what a pass cannot do without
def work(case):
    R, K, op = case["rows"], case["K"], case["op"]
    e = 4 if case["dtype"] == "f32" else 2
    if op == "round4":
        return {"bytes": 2.0 * e * R * K, "flops": 0.0}
    if op in ("norm", "norm8", "grad"):
        we = 4 if case["w"] == "f32" else 2
        if op == "grad":
            return {"bytes": e * R * K * (4.0 if case["residual"] else 3.0) + 2.0 * we * K, "flops": 8.0 * R * K}
        stream = e * R * K * (3.0 if case["residual"] else 1.0) + we * K  # x, r and h
        if op == "norm":
            return {"bytes": stream + e * R * K, "flops": 4.0 * R * K}
        return {"bytes": stream + case["N"] * (K + 4.0) + e * R * case["N"], "flops": 2.0 * R * case["N"] * K}
    N = case["N"]
    touched = float(np.sum(1.0 - (1.0 - np.minimum(_popularity(case), 1.0 - 1e-12)) ** R))  # groups with rows
    return {"bytes": e * ((case["tokens"] or R) * K + R * N) + touched * N * (K / 2 + K / 32), "flops": 2.0 * R * N * K}


# ----------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    """From the formulas in float64; rounded where the definition rounds (h, and the codes)."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "grad":  # y_i = w_i h_i / m, m = sqrt(mean h^2 + eps)
        h, dy, w = s["h"].double(), s["dy"].double(), s["weight"].double()
        m = (h.pow(2).sum(dim=1) / case["K"] + EPS).sqrt()[:, None]
        dot = (dy * w * h).sum(dim=1, keepdim=True)
        dx = dy * w / m - h * dot / (case["K"] * m ** 3)
        return dx if s["dh"] is None else dx + s["dh"].double(), (dy * h / m).sum(dim=0)
    if op in ("norm", "norm8"):
        h = s["x"].double()
        if s["r"] is not None:
            h = (h + s["r"].double()).to(s["x"].dtype).double()
        y = h * s["weight"].double() / (h.pow(2).sum(dim=1) / case["K"] + EPS).sqrt()[:, None]
        if op == "norm8":
            top = y.abs().max(dim=1).values[:, None]
            q = torch.round(127.0 * y / torch.where(top == 0, torch.ones_like(top), top))
            y = torch.matmul(q, s["wq"][0].double().t()) * (top / 127.0) * s["ws"][0].double()
        return y if op == "norm" and s["r"] is None else (y,) if s["r"] is None else (y, h)

    def power(e):  # 2^e
        return ((e.long() + 1023) << 52).view(torch.float64)

    def value(x):  # x in 64 bits -> what its 4-bit code stands for
        b = x.reshape(x.shape[0], -1, 32)
        top = b.abs().max(dim=2).values
        e = torch.where(top > 0, torch.frexp(top)[1] - 3, torch.full_like(top, -127, dtype=torch.int32)).clamp(min=-127)
        unit = power(e)[:, :, None]
        m = (b / unit).abs()
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
        return ((torch.round(m / step) * step).clamp(max=6.0) * unit * b.sign()).view(x.shape)

    if op == "round4":
        return torch.cat([value(p.double()) for p in s["x"].split(4096)])
    x = value(s["x"].double())
    if s["row_index"] is not None:
        x = x[s["row_index"].long()]
    grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], dtype=torch.float64, device="cuda") / 2
    both = torch.stack([grid.repeat(16), grid.repeat_interleave(16)], dim=1)  # byte -> (low, high)
    parts = []
    for g in range(len(s["ends"]) - 1):
        rows = slice(s["ends"][g], s["ends"][g + 1])
        if rows.start == rows.stop:
            continue
        unit = power(s["ws"][g][:, :case["K"] // 32].int() - 127)
        w = both[s["wq"][g].int()].view(case["N"], -1, 32) * unit[:, :, None]
        parts.append(torch.matmul(x[rows], w.view(case["N"], -1).t()))
    return torch.cat(parts)
