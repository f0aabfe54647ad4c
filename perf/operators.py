"""The grouped matrix products of an MoE layer, their gradients, and the 8-bit integer products, as a
user of the library calls them: what is run, on which inputs, and what each pass cannot do without.

A case names its operator in ``op``:

* ``gm``   the product of ragged row groups with their group's weight (moe_grouped_matmul)
* ``dx``   its gradient for the rows (moe_grouped_matmul_dx)
* ``dw``   its gradient for the weights (moe_grouped_matmul_dw)
* ``i8``   rows quantized to 8-bit integers on the fly, then the product with 8-bit weights
           (moe_quantize_rows, moe_matmul_i8), in one group or grouped
* ``ffn8`` a SwiGLU expert FFN in 8-bit integers: quantize, gate and up, SwiGLU and quantize, down

Sizes: ``G`` groups (``0``: one group, no offsets), ``rows`` over all groups, weights ``[G, N, K]``
(``ffn8``: hidden size ``K``, intermediate size ``N``), ``tokens`` > 0: the rows gather from that many
token rows.  ``spread`` says how the rows fall on the groups: ``even`` (a balanced router: multinomial),
``skew`` (popularity 1/rank^1.1, several groups empty), ``one`` (all in one group).

Where ``own`` is false the same values come from elementary torch operations in float32: the groups padded
to the largest one, one batched product, the rows taken out again.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
PAD_BYTES = 12e9     # a drawn case's padded operands and weights in float32, each
MOST_FLOPS = 1.5e12  # a drawn case's padded product


def listed():
    return [
        # the tiny fp32 layer of the tests and the benchmark: 64 tokens, top-2 of 16 experts; latency counts
        dict(name="gm_tiny_f32", op="gm", dtype="f32", G=16, rows=128, N=128, K=256, tokens=64, spread="even"),
        # decoding 64 tokens, top-8 of 384 experts: the down product, about one row per expert, weights streamed
        dict(name="gm_decode", op="gm", dtype="bf16", G=384, rows=512, N=7168, K=2048, tokens=0, spread="even"),
        # a prompt of 8192 tokens, top-8 of 384: the gate product on rows gathered from the tokens
        dict(name="gm_prefill", op="gm", dtype="bf16", G=384, rows=65536, N=2048, K=7168, tokens=8192, spread="even"),
        # one expert-parallel rank's share: 3 experts, 16384 rows, gate and up side by side
        dict(name="gm_share", op="gm", dtype="bf16", G=3, rows=16384, N=4096, K=7168, tokens=0, spread="even"),
        # the same share in training: the rows' gradient through gate and up
        dict(name="dx_share", op="dx", dtype="bf16", G=3, rows=16384, N=4096, K=7168, tokens=0, spread="even"),
        # a small fp32 layer of odd sizes, one expert taking most rows and some none: the rows' gradient
        dict(name="dx_odd_f32", op="dx", dtype="f32", G=9, rows=777, N=1001, K=515, tokens=0, spread="skew"),
        # the share's weight gradient: few experts, a long sum over rows
        dict(name="dw_share", op="dw", dtype="bf16", G=3, rows=16384, N=2048, K=7168, tokens=0, spread="even"),
        # an eighth of the experts on one GPU, 8192 rows: about 170 rows a sum, the gradients' writes count
        dict(name="dw_many", op="dw", dtype="bf16", G=48, rows=8192, N=7168, K=2048, tokens=0, spread="even"),
        # the dense first layer's gate at decode: 64 rows, one group, weights streamed as bytes
        dict(name="i8_decode", op="i8", dtype="bf16", G=0, rows=64, N=18432, K=7168, tokens=0, spread="one"),
        # the same layer on a prompt of 8192 tokens
        dict(name="i8_prefill", op="i8", dtype="bf16", G=0, rows=8192, N=18432, K=7168, tokens=0, spread="one"),
        # 64 tokens' gathered rows on 48 experts' gate, unevenly: some experts empty
        dict(name="i8_experts", op="i8", dtype="bf16", G=48, rows=512, N=2048, K=7168, tokens=64, spread="skew"),
        # 48 experts' whole FFN on 8192 rows
        dict(name="ffn8_experts", op="ffn8", dtype="bf16", G=48, rows=8192, N=2048, K=7168, tokens=0, spread="even"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, i8=False):
    """A matrix side: most often a multiple of 64 as models have them, sometimes of 8 (16 for the bytes of an
    8-bit row), sometimes anything."""
    v = _log(rng, lo, hi)
    step = rng.choice((64, 64, 64, 16 if i8 else 8, 1))
    return max(step, v // step * step)


def _popularity(case):
    G = max(1, case["G"])
    if case["spread"] == "skew":
        p = 1.0 / np.arange(1, G + 1) ** 1.1
    elif case["spread"] == "one":
        p = np.zeros(G)
        p[0] = 1.0
    else:
        p = np.ones(G)
    return p / p.sum()


def _padded_rows(case):
    """About how many rows the groups have when each is padded to the largest."""
    top = case["rows"] * _popularity(case).max()
    return max(1, case["G"]) * (top + 4 * math.sqrt(top) + 4)


def draw(rng):
    while True:
        op = rng.choice(("gm", "gm", "dx", "dx", "dw", "dw", "i8", "i8", "ffn8"))
        i8 = op in ("i8", "ffn8")
        G = _log(rng, 1, 384)
        if op == "i8" and rng.random() < 0.5:
            G = 0
        # 8-bit paths take bf16 rows here: their quotients 127 x / max|x| are then exact enough for every code to be
        # the same in 32 and in 64 bits
        case = dict(op=op, dtype="f32" if rng.random() < 0.25 and not i8 else "bf16", G=G, rows=_log(rng, 1, 65536),
                    N=_size(rng, 64, 18432 if op == "i8" else 7168, i8), K=_size(rng, 64, 7168, i8), tokens=0,
                    spread="one" if G == 0 else rng.choice(("even", "even", "skew")))
        if op in ("gm", "dw") and rng.random() < 0.3:
            case["tokens"] = max(1, case["rows"] // rng.choice((2, 4, 8)))
        if 3072 in (case["rows"], case["N"], case["K"], 2 * case["N"]):  # no size of this layer
            continue
        p, n = _padded_rows(case), max(1, G) * case["N"] * case["K"] * (3 if op == "ffn8" else 1)
        if 4 * n <= PAD_BYTES and 4 * p * max(case["N"] * (2 if op == "ffn8" else 1), case["K"]) <= PAD_BYTES \
                and 2 * p * case["N"] * case["K"] * (3 if op == "ffn8" else 1) <= MOST_FLOPS:
            return case


def _counts(case, seed):
    rng = np.random.default_rng([int(seed), 1])
    p = _popularity(case)
    if case["spread"] == "skew":
        p = rng.permutation(p)
    return rng.multinomial(case["rows"], p)


def _i8_weight(gen, shape):
    """Weights already stored in 8 bits: codes and each output channel's scale."""
    codes = torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
    scales = torch.rand(shape[:-1], generator=gen, device="cuda") * 0.5 + 0.75
    return codes, scales / (73.0 * math.sqrt(shape[-1]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, rows, N, K, op = DTYPES[case["dtype"]], case["rows"], case["N"], case["K"], case["op"]
    G = max(1, case["G"])

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dt).mul_(scale)

    counts = _counts(case, seed)
    s = dict(op=op, group_offsets=None, row_index=None, cap=int(counts.max()))
    if case["G"]:
        s["group_offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    if case["tokens"]:
        s["row_index"] = torch.randint(0, case["tokens"], (rows,), generator=gen, device="cuda", dtype=torch.int32)
    if op in ("gm", "dw", "i8", "ffn8"):
        s["x"] = normal(case["tokens"] or rows, K)
    if op in ("dx", "dw"):
        s["dy"] = normal(rows, N)
    if op in ("gm", "dx"):
        s["w"] = normal(G, N, K, scale=1.0 / math.sqrt(K if op == "gm" else N))
    if op in ("i8", "ffn8"):  # activations have a few large channels
        s["x"][:, torch.randperm(K, generator=gen, device="cuda")[:max(1, K // 100)]] *= 6.0
    if op == "i8":
        s["w"], s["w_scale"] = _i8_weight(gen, (G, N, K))
    if op == "ffn8":
        s["w"], s["w_scale"] = _i8_weight(gen, (G, 2 * N, K))  # gate rows, then up rows
        s["w_down"], s["w_down_scale"] = _i8_weight(gen, (G, K, N))
    return s


# ----------------------------------------------------------------- the library's operators
def _own(s):
    import moe_layer_forward_amd as moe

    op, off, idx = s["op"], s["group_offsets"], s["row_index"]
    if op == "gm":
        return moe.moe_grouped_matmul(s["x"], s["w"], off, row_index=idx)
    if op == "dx":
        return moe.moe_grouped_matmul_dx(s["dy"], s["w"], off)
    if op == "dw":
        return moe.moe_grouped_matmul_dw(s["dy"], s["x"], off, row_index=idx)
    q, sq = moe.moe_quantize_rows(s["x"])
    y_dtype = moe.MOE_BF16 if s["x"].dtype == torch.bfloat16 else moe.MOE_F32
    if op == "i8":
        return moe.moe_matmul_i8(q, sq, s["w"], s["w_scale"], off, row_index=idx, y_dtype=y_dtype)
    gate_up = moe.moe_matmul_i8(q, sq, s["w"], s["w_scale"], off, y_dtype=moe.MOE_F32)
    h, sh = moe.moe_quantize_rows(gate_up, swiglu=True)
    return moe.moe_matmul_i8(h, sh, s["w_down"], s["w_down_scale"], off, y_dtype=y_dtype)


# ----------------------------------------------------------------- the plain forms
def _slots(s, rows, G):
    """Row r's place in the groups padded to the largest, [G * cap] rows."""
    r = torch.arange(rows, device="cuda")
    if s["group_offsets"] is None:
        return r
    off = s["group_offsets"].long()
    g = torch.searchsorted(off[1:], r, right=True)
    return g * s["cap"] + (r - off[g])


def _pad(v, slots, G, cap):
    out = torch.zeros((G * cap, v.shape[1]), device="cuda")
    out[slots] = v
    return out.view(G, cap, v.shape[1])


def _product(v, w, slots, cap):
    """[rows, N] = v [rows, K] times each row's group of w [G, N, K], float32."""
    G, N, K = w.shape
    if G == 1:
        return v @ w[0].t()
    p = torch.bmm(w, _pad(v, slots, G, cap).transpose(1, 2).contiguous())  # [G, N, cap]
    return p.transpose(1, 2).reshape(G * cap, N)[slots]


def _quantized(v):
    a = v.abs().amax(dim=1, keepdim=True)
    return torch.where(a > 0, torch.round(v * 127.0 / a), torch.zeros_like(v)), a[:, 0] / 127.0


def _row_scales(w_scale, slots, cap):
    """Each row's group's channel scales, [rows, N]."""
    return w_scale[0] if w_scale.shape[0] == 1 else w_scale[slots // cap]


def _plain(s):
    op = s["op"]
    w = s["w"].float() if "w" in s else None
    rows = s["dy"].shape[0] if "dy" in s else s["x"].shape[0] if s["row_index"] is None else s["row_index"].shape[0]
    G = w.shape[0] if w is not None else s["group_offsets"].shape[0] - 1
    slots, cap = _slots(s, rows, G), max(1, s["cap"])
    x = s["x"].float() if "x" in s else None
    if op == "gm":
        x = x if s["row_index"] is None else x[s["row_index"].long()]
        return _product(x, w, slots, cap).to(s["x"].dtype)
    if op == "dx":
        return torch.bmm(_pad(s["dy"].float(), slots, G, cap), w).view(G * cap, -1)[slots].to(s["dy"].dtype)
    if op == "dw":
        x = x if s["row_index"] is None else x[s["row_index"].long()]
        dyt = _pad(s["dy"].float(), slots, G, cap).transpose(1, 2).contiguous()
        return torch.bmm(dyt, _pad(x, slots, G, cap)).to(s["dy"].dtype)
    q, sq = _quantized(x)
    if s["row_index"] is not None:
        q, sq = q[s["row_index"].long()], sq[s["row_index"].long()]
    y = _product(q, w, slots, cap) * sq[:, None] * _row_scales(s["w_scale"], slots, cap)
    if op == "i8":
        return y.to(s["x"].dtype)
    n = y.shape[1] // 2
    h, sh = _quantized(y[:, :n] / (1.0 + torch.exp(-y[:, :n])) * y[:, n:])
    y = _product(h, s["w_down"].float(), slots, cap) * sh[:, None] * _row_scales(s["w_down_scale"], slots, cap)
    return y.to(s["x"].dtype)


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------- what a pass cannot do without
def work(case):
    G, R, N, K = max(1, case["G"]), case["rows"], case["N"], case["K"]
    e, T = 4 if case["dtype"] == "f32" else 2, case["tokens"] or case["rows"]
    touched = float(np.sum(1.0 - (1.0 - np.minimum(_popularity(case), 1.0 - 1e-12)) ** R))  # groups with rows
    flops = 2.0 * R * N * K
    if case["op"] == "gm":
        return {"bytes": e * (T * K + touched * N * K + R * N), "flops": flops}
    if case["op"] == "dx":
        return {"bytes": e * (R * N + touched * N * K + R * K), "flops": flops}
    if case["op"] == "dw":
        return {"bytes": e * (R * N + T * K + G * N * K), "flops": flops}
    if case["op"] == "i8":
        return {"bytes": e * (T * K + R * N) + touched * N * (K + 4), "flops": flops}
    return {"bytes": e * 2 * R * K + touched * (3 * N * K + 4 * (2 * N + K)), "flops": 3 * flops}


# ----------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    """Group by group from the formulas, in float64; the quantizer's codes too (a tie goes to the even code)."""
    s = prepare(case, seed)
    op, R = case["op"], case["rows"]
    ends = [0, R] if s["group_offsets"] is None else s["group_offsets"].cpu().tolist()
    src = torch.arange(R, device="cuda") if s["row_index"] is None else s["row_index"].long()

    def codes(v):
        top = v.abs().max(dim=1).values
        return torch.round(127.0 * v / torch.where(top == 0, torch.ones_like(top), top)[:, None]), top / 127.0

    parts = []
    for g in range(len(ends) - 1):
        r = slice(ends[g], ends[g + 1])
        if op == "gm":
            parts.append(torch.matmul(s["x"][src[r]].double(), s["w"][g].double().t()))
        elif op == "dx":
            parts.append(torch.matmul(s["dy"][r].double(), s["w"][g].double()))
        elif op == "dw":
            parts.append(torch.matmul(s["dy"][r].double().t(), s["x"][src[r]].double()))
        else:
            if ends[g] == ends[g + 1]:
                continue
            q, sq = codes(s["x"][src[r]].double())
            y = torch.matmul(q, s["w"][g].double().t()) * sq[:, None] * s["w_scale"][g].double()
            if op == "ffn8":
                gate, up = y.chunk(2, dim=1)
                q, sq = codes(gate * torch.sigmoid(gate) * up)
                y = torch.matmul(q, s["w_down"][g].double().t()) * sq[:, None] * s["w_down_scale"][g].double()
            parts.append(y)
    return torch.stack(parts) if op == "dw" else torch.cat(parts)
