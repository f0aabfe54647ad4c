"""Microscaled 4-bit floating point: rows to codes and back, and the grouped product, against float64.

The oracle is numpy on the CPU, written from include/moe.h."""
import ctypes

import numpy as np
import pytest

import moe_layer_forward_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _torch():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _oracle_quantize(v):
    """(codes [rows, K], scale powers [rows, K / 32]) of float64 rows."""
    b = v.reshape(v.shape[0], -1, 32)
    with np.errstate(invalid="ignore"):
        a = np.abs(b).max(axis=2)
    ok = np.isfinite(b).all(axis=2)
    e = np.frexp(np.where(ok, a, 1.0))[1] - 1  # floor(log2 a)
    s = np.where(a == 0, 0, np.maximum(e - 2, -127) + 127)
    m = np.abs(np.where(ok[..., None], b, 0.0)) * 2.0 ** (127.0 - s)[..., None]
    c = sum((m > t if k % 2 == 0 else m >= t).astype(int) for k, t in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    c = np.where(ok[..., None], c + 8 * np.signbit(b), 0)
    return c.reshape(v.shape), np.where(ok, s, 255)


def _unpack(codes):
    c = codes.cpu().numpy()
    return np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:-1], 2 * c.shape[-1]).astype(int)


def _values(codes, scales):
    """float64 values of packed codes [.., K / 2] and scales."""
    c = _unpack(codes)
    K = c.shape[-1]
    s = scales.cpu().numpy()[..., :K // 32].astype(int)
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    unit = np.where(s == 255, np.nan, 2.0 ** (s - 127.0))
    return v * np.repeat(unit, 32, axis=-1)


def _rows(rows, K, seed, dt="bf16"):
    torch = _torch()
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-20, 20, (rows, K // 32))).repeat(32, axis=1)
    return torch.from_numpy(x).to("cuda", {"bf16": torch.bfloat16, "f32": torch.float32}[dt])


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (5, 480), (2, 512), (7, 544), (65, 7168), (700, 2048), (40000, 64), (9, 64), (13, 128), (31, 160), (1001, 256), (17, 224), (4099, 32)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_codes_are_those_of_the_formula(rows, K, dt):
    x = _rows(rows, K, rows, dt)
    codes, scales = moe.moe_quantize_mx4(x)
    c, s = _oracle_quantize(x.double().cpu().numpy())
    assert (_unpack(codes) == c).all()
    got = scales.cpu().numpy()
    assert got.shape == (rows, moe.mx4_scale_cols(K)) and (got[:, :K // 32] == s).all() and not got[:, K // 32:].any()
    for y_dtype, t in ((moe.MOE_BF16, "bfloat16"), (moe.MOE_F32, "float32")):
        y = moe.moe_dequantize_mx4(codes, scales, y_dtype)
        assert str(y.dtype) == f"torch.{t}" and (y.double().cpu().numpy() == _values(codes, scales)).all()


def test_ties_borders_and_extremes():
    """Every tie and its neighbours at every scale a type reaches, signs of zero, subnormals, the largest values."""
    torch = _torch()
    marks = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    for dt, low, high in (("bfloat16", -130, 124), ("float32", -147, 124)):
        t = getattr(torch, dt)
        rows = []
        for p in range(low, high):
            v = torch.from_numpy(np.concatenate([marks, -marks]) * 2.0 ** p).to(t)
            one = torch.tensor([1 if i % 2 else -1 for i in range(32)], dtype=torch.int32)
            raw = v.view(torch.int16 if t == torch.bfloat16 else torch.int32)
            near = torch.where(v == 0, raw, raw + one.to(raw.dtype)).view(t)
            rows += [v, near]
        x = torch.stack(rows).cuda()
        codes, scales = moe.moe_quantize_mx4(x)
        c, s = _oracle_quantize(x.double().cpu().numpy())
        assert (scales.cpu().numpy()[:, :1] == s).all() and (_unpack(codes) == c).all()
        big = torch.full((1, 32), torch.finfo(t).max, dtype=t, device="cuda")
        codes, scales = moe.moe_quantize_mx4(big)
        assert int(scales[0, 0]) == 252 and (_unpack(codes) == 7).all()


def test_blocks_with_infinities_nan_and_zeros():
    torch = _torch()
    x = _rows(4, 1024, 1)
    clean = moe.moe_quantize_mx4(x)
    x[1, 40], x[2, 0], x[3, 1023] = float("inf"), float("nan"), float("-inf")
    x[0, 64:96] = 0
    codes, scales = moe.moe_quantize_mx4(x)
    c, s = _oracle_quantize(x.double().cpu().numpy())
    assert (_unpack(codes) == c).all() and (scales.cpu().numpy() == s).all()
    assert int(scales[1, 1]) == int(scales[2, 0]) == int(scales[3, 31]) == 255 and int(scales[0, 2]) == 0
    assert bool((scales == clean[1]).sum() == scales.numel() - 4)
    y = moe.moe_dequantize_mx4(codes, scales, moe.MOE_F32).cpu().numpy()
    assert np.isnan(y).sum() == 3 * 32 and not y[0, 64:96].any()
    # the ends of the scales: 2^-127 (subnormal values) and 2^127 (6 2^127 is past fp32: infinite)
    codes = torch.tensor([[0x71] * 16, [0x71] * 16], dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, 16), dtype=torch.uint8, device="cuda")
    scales[1, 0] = 254
    y = moe.moe_dequantize_mx4(codes, scales, moe.MOE_F32).double().cpu().numpy()
    assert (y[0, 0::2] == 2.0 ** -128).all() and (y[0, 1::2] == 6 * 2.0 ** -127).all()
    assert (y[1, 0::2] == 2.0 ** 126).all() and np.isinf(y[1, 1::2]).all()


@pytest.mark.parametrize("rows,cols", [(3, 32), (50, 2048), (9, 992), (37, 64), (21, 96), (19, 256)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_swiglu_before_the_codes(rows, cols, dt):
    """v = SiLU(g) u in fp32 (expf, a sum, a division, two products: 2^-20 relative); a code is the nearest value's but
    where v is that near to a tie, a scale that of the largest value but where it is that near to a power of two."""
    torch = _torch()
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(rng.standard_normal((rows, 2 * cols)) * 2).to("cuda", torch.bfloat16 if dt == "bf16" else torch.float32)
    codes, scales = moe.moe_quantize_mx4(x, swiglu=True)
    g, u = np.split(x.double().cpu().numpy(), 2, axis=1)
    v = g / (1 + np.exp(-g)) * u
    lo, hi = _oracle_quantize(v * (1 - 2.0 ** -20)), _oracle_quantize(v * (1 + 2.0 ** -20))
    s, c = scales.cpu().numpy()[:, :cols // 32], _unpack(codes)
    same = (lo[1] == hi[1])
    assert ((s == lo[1]) | (s == hi[1])).all() and same.mean() > 0.99
    same = same.repeat(32, axis=1)
    assert ((c == lo[0]) | (c == hi[0]) | ~same).all()


def test_swiglu_of_far_gates():
    """SiLU where its exponential is tiny, huge and past the type's range; infinities and NaN; tiny and huge factors."""
    torch = _torch()
    g = np.array([-88.5, -80.25, -64.0, -44.5, -20.0, -1e-3, -1e-30, 1e-30, 0.5, 17.0, 88.0, 89.5, 120.0, 1e4, 1e30])
    for factor in (1.0, 2.0 ** 60, 2.0 ** -20):
        x = np.concatenate([np.repeat(g[:, None], 32, axis=1), np.full((len(g), 32), factor)], axis=1).astype(np.float32)
        codes, scales = moe.moe_quantize_mx4(torch.from_numpy(x).cuda(), swiglu=True)
        v = x[:, :32].astype(np.float64)
        v = v / (1 + np.exp(-v)) * factor
        some = (np.abs(v[:, 0]) < 2.0 ** 127) & (np.abs(v[:, 0]) > 2.0 ** -125)
        got = _values(codes, scales)
        # the nearest code of a block of one value in [4, 8) units: within a unit of it below 6, two above
        assert (np.abs(got - v)[some] <= np.abs(v)[some] * (0.25 + 2.0 ** -20)).all()
        lo, hi = _oracle_quantize(v * (1 - 2.0 ** -20)), _oracle_quantize(v * (1 + 2.0 ** -20))
        c, s = _unpack(codes), scales.cpu().numpy()[:, :1]
        same = lo[1] == hi[1]
        assert (((c == lo[0]) | (c == hi[0]))[(same & some[:, None])[:, 0]]).all() and ((s == lo[1]) | (s == hi[1]))[some].all()
    for gate, up, nan in ((-1e4, 1.0, False), (-200.0, -3.0, False), (float("inf"), 1.0, True), (float("nan"), 1.0, True), (1.0, float("inf"), True),
                          (0.0, float("nan"), True), (0.0, 5.0, False)):
        x = torch.zeros((1, 64), device="cuda")
        x[0, 3], x[0, 35] = gate, up
        codes, scales = moe.moe_quantize_mx4(x, swiglu=True)
        assert int(scales[0, 0]) == (255 if nan else 0) and not bool((_unpack(codes) & 7).any())


def test_rows_that_start_anywhere():
    torch = _torch()
    for t in (torch.bfloat16, torch.float32):
        flat = torch.randn(5 * 96 + 1, device="cuda").to(t)
        x = flat[1:].view(5, 96)
        a, b = moe.moe_quantize_mx4(x), moe.moe_quantize_mx4(x.clone())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        out = torch.zeros(5 * 96 + 1, device="cuda", dtype=t)[1:].view(5, 96)
        assert torch.equal(moe.moe_dequantize_mx4(*a, out=out), moe.moe_dequantize_mx4(*a, out=torch.empty_like(x)))


# ------------------------------------------------------------------------------------------------ the product
def _weights(G, N, K, seed):
    torch = _torch()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    codes = torch.randint(0, 256, (G, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(117, 134, (G, N, moe.mx4_scale_cols(K)), generator=gen, device="cuda", dtype=torch.uint8)
    return codes, scales


def _check_product(y, xc, xs, wc, ws, sizes, index=None, past=0):
    """Sums of K / 128 matrix instructions, each off by at most u of its terms' magnitudes and the addition by u of the
    sum so far, then up to 16 joined ranges: (K / 128 + 20) 2 u of the magnitudes, and the output's rounding."""
    torch = _torch()
    x, K = torch.from_numpy(_values(xc, xs)), xc.shape[1] * 2
    if index is not None:
        x = x[index.cpu().long()]
    half = 2.0 ** -8 if y.dtype == torch.bfloat16 else U
    at = 0
    for g, n in enumerate(sizes):
        if n:
            w = torch.from_numpy(_values(wc[g], ws[g]))
            rows = x[at:at + n]
            ref, mag = rows @ w.T, rows.abs() @ w.abs().T
            err = (y[at:at + n].double().cpu() - ref).abs()
            bound = (K / 128 + 20) * 2 * U * mag + half * ref.abs() + 2.0 ** -126
            assert bool((err <= bound).all()), (g, float((err / bound).max()))
        at += n
    assert at + past == len(y)


def _offsets(sizes):
    torch = _torch()
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


SIZES = ([1], [0, 3, 0, 17], [16, 1, 15, 0], [64, 65, 63, 1], [300, 0, 5], [128, 256, 257], [511], [0, 0], [700, 1100, 3])


@pytest.mark.parametrize("sizes", SIZES, ids=["-".join(map(str, s)) for s in SIZES])
@pytest.mark.parametrize("N,K", [(1, 32), (65, 96), (64, 512), (130, 544), (257, 1024), (300, 2080)])
@pytest.mark.parametrize("y_dtype", [moe.MOE_BF16, moe.MOE_F32], ids=["bf16", "f32"])
def test_products_of_groups(sizes, N, K, y_dtype):
    rows, G = sum(sizes), len(sizes)
    xc, xs = moe.moe_quantize_mx4(_rows(rows, K, 1))
    wc, ws = _weights(G, N, K, 2)
    y = moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes), y_dtype=y_dtype)
    assert y.shape == (rows, N)
    _check_product(y, xc, xs, wc, ws, sizes)


@pytest.mark.parametrize("rows,N,K", [(1, 64, 7168), (1, 2048, 18432), (16, 512, 7168), (17, 7168, 2048), (64, 1000, 7168),
                                      (100, 4096, 512), (513, 520, 4128), (2000, 768, 1536), (1, 1, 32), (33, 16384, 64),
                                      (9, 33, 65536)])
def test_one_group(rows, N, K):
    xc, xs = moe.moe_quantize_mx4(_rows(rows, K, 3))
    wc, ws = _weights(1, N, K, 4)
    _check_product(moe.moe_matmul_mx4(xc, xs, wc, ws, y_dtype=moe.MOE_F32), xc, xs, wc, ws, [rows])


@pytest.mark.parametrize("rows", [5, 70, 400, 3000])
def test_whole_numbers_are_exact(rows):
    """Scales 1 and sums below 2^24 / 4 quarters: every sum is a multiple of 1/4 that fp32 holds."""
    torch = _torch()
    K, N, sizes = 1536, 200, [rows // 3, 0, rows - rows // 3]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    xc = torch.randint(0, 256, (rows, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    wc = torch.randint(0, 256, (3, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    xs = torch.full((rows, moe.mx4_scale_cols(K)), 127, dtype=torch.uint8, device="cuda")
    ws = torch.full((3, N, moe.mx4_scale_cols(K)), 127, dtype=torch.uint8, device="cuda")
    y = moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes), y_dtype=moe.MOE_F32).double().cpu()
    x, w = torch.from_numpy(_values(xc, xs)), torch.from_numpy(_values(wc, ws))
    ref = torch.cat([x[:sizes[0]] @ w[0].T, x[sizes[0]:] @ w[2].T])
    assert torch.equal(y, ref)


@pytest.mark.parametrize("tokens,rows", [(1, 9), (40, 64), (64, 900), (500, 4000)])
def test_gathered_rows(tokens, rows):
    """Rows named several times, in any order; rows past the last group stay as they were."""
    torch = _torch()
    N, K, past = 96, 1056, 7
    sizes = [rows // 2, 0, rows - rows // 2 - 1, 1]
    xc, xs = moe.moe_quantize_mx4(_rows(tokens, K, 5))
    wc, ws = _weights(4, N, K, 6)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    index = torch.randint(0, tokens, (rows + past,), generator=gen, device="cuda", dtype=torch.int32)
    out = torch.full((rows + past, N), 77.0, device="cuda")
    y = moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes), row_index=index, out=out)
    assert y is out and bool((out[rows:] == 77).all())
    _check_product(y, xc, xs, wc, ws, sizes, index, past)
    # rows that are not in x are moved inside: nothing past x is read
    index[::3] = tokens + 5
    index[1::3] = -4
    y = moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes), row_index=index)
    assert bool(torch.isfinite(y[:rows].float()).all())


@pytest.mark.parametrize("rows", [3, 200, 1500])
def test_nan_stays_in_its_row_and_column_and_padding_is_not_read(rows):
    torch = _torch()
    N, K = 90, 1120  # 35 blocks of 48
    xc, xs = moe.moe_quantize_mx4(_rows(rows, K, 7))
    wc, ws = _weights(1, N, K, 8)
    want = moe.moe_matmul_mx4(xc, xs, wc, ws, y_dtype=moe.MOE_F32)
    xs[:, 35:] = 255
    ws[:, :, 35:] = 255
    assert torch.equal(moe.moe_matmul_mx4(xc, xs, wc, ws, y_dtype=moe.MOE_F32), want)
    xs[rows // 2, 34] = 255
    ws[0, 40, 0] = 255
    y = moe.moe_matmul_mx4(xc, xs, wc, ws, y_dtype=moe.MOE_F32)
    assert bool(y[rows // 2].isnan().all()) and bool(y[:, 40].isnan().all())
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[rows // 2], keep[:, 40] = False, False
    assert torch.equal(y[keep], want[keep])


def test_skewed_groups_and_the_same_bits_every_time():
    torch = _torch()
    sizes = [900, 0, 1, 2, 0, 40, 17, 64, 0, 3] + [1] * 30
    xc, xs = moe.moe_quantize_mx4(_rows(sum(sizes), 2048, 9))
    wc, ws = _weights(len(sizes), 264, 2048, 10)
    y = moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes))
    _check_product(y, xc, xs, wc, ws, sizes)
    for _ in range(3):
        assert torch.equal(moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes)), y)


def test_many_groups():
    sizes = np.random.default_rng(1).multinomial(512, np.ones(384) / 384).tolist()
    xc, xs = moe.moe_quantize_mx4(_rows(512, 1024, 11))
    wc, ws = _weights(384, 136, 1024, 12)
    _check_product(moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes)), xc, xs, wc, ws, sizes)


@pytest.mark.parametrize("rows", [9, 600])
def test_another_stream_and_a_captured_graph(rows):
    """An expert's FFN in this format, replayed with new inputs in between, against eager calls."""
    torch = _torch()
    H, inner, G = 512, 288, 3
    x = _rows(rows, H, 13) * 2.0 ** -10
    off = _offsets([rows // 3, 0, rows - rows // 3])
    gate_up, down = _weights(G, 2 * inner, H, 14), _weights(G, H, inner, 15)

    def run():
        q = moe.moe_quantize_mx4(x)
        h = moe.moe_quantize_mx4(moe.moe_matmul_mx4(*q, *gate_up, off, y_dtype=moe.MOE_F32), swiglu=True)
        return moe.moe_matmul_mx4(*h, *down, off)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = run()
    side.synchronize()
    assert torch.equal(first, run())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in range(4):
        x.copy_(_rows(rows, H, 20 + seed) * 2.0 ** -10)
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.nan_to_num(), want.nan_to_num())


def test_two_streams_and_two_graphs_of_one_workspace():
    """Products with packed scales: at once on two streams, and captured twice with the same workspace, replayed in turn."""
    torch = _torch()
    x = [moe.moe_quantize_mx4(_rows(8192, 4096, 31 + i)) for i in range(2)]
    w = [_weights(1, 4608, 4096, 33 + i) for i in range(2)]
    want = [moe.moe_matmul_mx4(*x[i], *w[i]) for i in range(2)]
    nbytes = moe.moe_matmul_workspace_size(moe.MOE_MATMUL_MX4, moe.MOE_F32, 1, 8192, 4608, 4096)
    assert nbytes > 0
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                got[i].append(moe.moe_matmul_mx4(*x[i], *w[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    graphs, out = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            out.append(moe.moe_matmul_mx4(*x[i], *w[i], workspace=ws))
    for _ in range(3):
        for i in range(2):
            out[i].fill_(7)
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[i], want[i]) for i in range(2))


def test_norm_experts_and_combine_together():
    """A layer as it would be served: residual and norm, routing, experts in this format, combine.  Every stage against
    float64 on the stage before, so that no code depends on a rounding that came earlier."""
    torch = _torch()
    T, H, I, E, K = 48, 256, 128, 8, 2
    cfg = moe.make_config(H, I, E, K, n_shared_experts=0)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    bf = lambda *s, scale=1.0: (torch.randn(s, generator=gen, device="cuda") * scale).bfloat16()  # noqa: E731
    x, res, wn, wr = bf(T, H), bf(T, H), bf(H, scale=0.1) + 1, bf(E, H, scale=0.02)
    gu, dn = moe.moe_quantize_mx4(bf(E * 2 * I, H, scale=H ** -0.5)), moe.moe_quantize_mx4(bf(E * H, I, scale=I ** -0.5))
    gu, dn = [t.view(E, 2 * I, -1) for t in gu], [t.view(E, H, -1) for t in dn]
    y, h = moe.moe_rms_norm(x, wn, residual=res)
    ids, weights = moe.moe_route(cfg, y, wr)
    off, row_token, pair_row, _ = moe.moe_permute(cfg, ids)
    sizes = (off[1:] - off[:-1]).tolist()
    q = moe.moe_quantize_mx4(y)
    mid = moe.moe_matmul_mx4(*q, *gu, off, row_index=row_token, y_dtype=moe.MOE_F32)
    _check_product(mid, *q, *gu, sizes, row_token)
    qm = moe.moe_quantize_mx4(mid, swiglu=True)
    rows = moe.moe_matmul_mx4(*qm, *dn, off)
    _check_product(rows, *qm, *dn, sizes)
    out = moe.moe_combine(cfg, rows, pair_row, weights)
    ref = (rows.double()[pair_row.long()] * weights.double()[:, :, None]).sum(dim=1)
    assert bool(((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 4 * U * 8).all())
    yref = h.double() / ((h.double() ** 2).mean(dim=1, keepdim=True) + 1e-6).sqrt() * wn.double()
    assert bool(((y.double() - yref).abs() <= (2.0 ** -8 + 40 * U) * yref.abs()).all())
    # and near the layer in 32 bits: 4-bit values are off by a tenth of a block's largest
    full = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    v = lambda t: torch.from_numpy(_values(*t)).cuda()  # noqa: E731
    wg, wd = v(gu), v(dn)
    for t in range(T):
        for k in range(K):
            e = int(ids[t, k])
            g, u = (wg[e] @ yref[t]).chunk(2)
            full[t] += float(weights[t, k]) * (wd[e] @ (g / (1 + torch.exp(-g)) * u))
    assert float((out.double() - full).norm() / full.norm()) < 0.35


def test_refusals():
    torch = _torch()
    xc, xs = moe.moe_quantize_mx4(_rows(4, 64, 1))
    wc, ws = _weights(2, 8, 64, 1)
    off = _offsets([2, 2])
    f = torch.zeros((4, 64), device="cuda")
    for bad in (lambda: moe.moe_quantize_mx4(f[:, :48].contiguous()), lambda: moe.moe_quantize_mx4(f.half()),
                lambda: moe.moe_quantize_mx4(f[:, ::2]), lambda: moe.moe_quantize_mx4(f, codes=xc[:2]),
                lambda: moe.moe_quantize_mx4(f, scales=xs[:, :2].contiguous()), lambda: moe.moe_quantize_mx4(f[0]),
                lambda: moe.moe_dequantize_mx4(xc, xs[:, :2].contiguous()), lambda: moe.moe_dequantize_mx4(xc.float(), xs),
                lambda: moe.moe_matmul_mx4(xc, xs, wc, ws), lambda: moe.moe_matmul_mx4(xc, xs, wc, ws, off.long()),
                lambda: moe.moe_matmul_mx4(xc, xs, wc[:, :, :16].contiguous(), ws, off),
                lambda: moe.moe_matmul_mx4(xc, xs[:3], wc, ws, off), lambda: moe.moe_matmul_mx4(xc.cpu(), xs, wc, ws, off),
                lambda: moe.moe_matmul_mx4(xc, xs, wc, ws, off, row_index=off.long()),
                lambda: moe.moe_matmul_mx4(xc, xs, wc, ws, off, out=f)):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros(4 * 32 + 8, dtype=torch.uint8, device="cuda")[8:].view(4, 32)
    with pytest.raises(moe.MoeError):
        moe.moe_matmul_mx4(odd, xs, wc, ws, off)


def test_large_matrices_to_codes_and_back():
    """Sizes that move with the non-temporal policy, four windows to a wave: the same codes as in parts."""
    torch = _torch()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    for rows, cols, swiglu in ((9001, 4640, False), (6000, 3520, True), (70001, 32, False)):
        x = torch.randn((rows, cols * (2 if swiglu else 1)), generator=gen, device="cuda").bfloat16()
        codes, scales = moe.moe_quantize_mx4(x, swiglu=swiglu)
        for a in range(0, rows, 1000):
            c, s = moe.moe_quantize_mx4(x[a:a + 1000], swiglu=swiglu)
            assert torch.equal(codes[a:a + 1000], c) and torch.equal(scales[a:a + 1000], s)
        if not swiglu:
            c, s = _oracle_quantize(x[-300:].double().cpu().numpy())
            assert (_unpack(codes[-300:]) == c).all() and (scales[-300:, :cols // 32].cpu().numpy() == s).all()
        y = moe.moe_dequantize_mx4(codes, scales)
        for a in range(0, rows, 1000):
            assert torch.equal(y[a:a + 1000], moe.moe_dequantize_mx4(codes[a:a + 1000], scales[a:a + 1000]))
        assert (y[-300:].double().cpu().numpy() == _values(codes[-300:], scales[-300:])).all()


def _exact_product(sizes, N, K, index_rows=0, seed=1):
    """Products of whole quarters: every sum is held by fp32, so that any kernel and order has to give it exactly."""
    torch = _torch()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rows, G = sum(sizes), len(sizes)
    x_rows = index_rows or rows
    xc = torch.randint(0, 256, (x_rows, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    wc = torch.randint(0, 256, (G, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    xs = torch.randint(126, 129, (x_rows, moe.mx4_scale_cols(K)), generator=gen, device="cuda", dtype=torch.uint8)
    ws = torch.randint(126, 129, (G, N, moe.mx4_scale_cols(K)), generator=gen, device="cuda", dtype=torch.uint8)
    index = torch.randint(0, x_rows, (rows,), generator=gen, device="cuda", dtype=torch.int32) if index_rows else None
    out = torch.full((rows + 5, N), 9.0, device="cuda")
    full = torch.cat([index, index[:5]]) if index_rows else None
    if not index_rows:
        xc, xs = torch.cat([xc, xc[:5]]), torch.cat([xs, xs[:5]])
    y = moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes), row_index=full, out=out)
    assert bool((y[rows:] == 9).all())
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    grid = torch.cat([grid, -grid])

    def values(c, s):
        v = grid[torch.stack([c & 15, c >> 4], dim=-1).int()].view(*c.shape[:-1], K // 32, 32)
        return (v * (2.0 * s[..., :K // 32].eq(128) + s[..., :K // 32].eq(127) + 0.5 * s[..., :K // 32].eq(126))[..., None]).view(*c.shape[:-1], K)

    x = values(xc, xs)
    x = x[full.long()] if index_rows else x
    at = 0
    for g, n in enumerate(sizes):
        if n:
            ref = x[at:at + n].double() @ values(wc[g], ws[g]).double().T
            assert torch.equal(y[at:at + n].double(), ref), g
        at += n


@pytest.mark.parametrize("sizes,N,K,index_rows", [
    ([8192], 4608, 4096, 0),                       # 256 x 256 tiles, packed scales
    ([6111], 5103, 6176, 700),                     # the same, gathered, odd sizes, the last window's padding
    ([3000, 0, 2500, 2777], 5120, 6048, 0),        # several groups packed
    ([2048], 8192, 7168, 0),
    ([5000], 2048, 1056, 0),                       # 128 x 128 tiles, few of them
    ([40000], 320, 1504, 0),                       # 128 x 128 tiles by the columns' padding, many row tiles
    ([100] * 40, 1100, 992, 0),                    # 128 x 128 tiles of groups
    ([200, 0, 300, 17, 1] * 9, 1000, 1024, 999),   # the same, gathered
    ([250, 0, 300, 17, 1, 400] * 12, 2048, 1056, 999),  # 256 x 256 tiles of groups, gathered
    ([130, 0, 257, 300, 5] * 8, 2048, 7168, 0),    # the same, weights read past the caches
    ([64, 0, 100, 1] * 10, 2048, 7168, 77),        # 128 x 128 tiles, the same
    ([150, 200] * 300, 512, 544, 0),               # more groups than are sorted
    ([5, 256, 31, 33, 0, 224, 255, 257, 511, 64, 1, 129] * 3, 1536, 2080, 0),  # every size of partial tile
    ([3, 0, 12, 1, 1, 7] * 40, 900, 1184, 0),      # the ring over groups of few rows
    ([1] * 300 + [0] * 300 + [30] * 100, 520, 544, 50),  # more than 512 groups, gathered
    ([5, 0, 2], 640, 6016, 0),                     # the stream kernel over groups
    ([7], 1025, 9216, 0), ([33], 5125, 4096, 0), ([20], 8200, 2080, 31), ([64], 5120, 1024, 0), ([50], 130, 8192, 0),
    ([64], 18432, 1024, 0),
    ([61], 18432, 2080, 0), ([128], 2048, 7168, 90), ([5, 0, 100, 64, 1], 700, 2336, 0), ([33], 9300, 2272, 0),
    ([128] * 7, 1100, 2048, 0), ([5], 28672, 512, 0), ([300], 1500, 2560, 0), ([129, 17, 128], 1024, 16416, 11),
])
def test_exact_sums_on_every_kernel(sizes, N, K, index_rows):
    _exact_product(sizes, N, K, index_rows)


def test_the_kernels_that_sizes_call_for():
    """The names the profile reports (include/moe.h), so that the cases above reach every kernel."""
    torch = _torch()
    hip = ctypes.CDLL("libamdhip64.so")
    events = (ctypes.c_void_p * 8)()
    for i in range(8):
        e = ctypes.c_void_p()
        assert hip.hipEventCreate(ctypes.byref(e)) == 0
        events[i] = e
    try:
        for sizes, N, K, want in (([8192], 4608, 4096, ["matmul_mx4_pack", "matmul_mx4_tile256"]), ([6111], 5103, 6176, ["matmul_mx4_pack", "matmul_mx4_tile256"]),
                                  ([3000, 0, 2500, 2777], 5120, 6048, ["matmul_mx4_pack", "matmul_mx4_tile256"]), ([40000], 320, 1504, ["matmul_mx4_tile128"]),
                                  ([300] * 50, 1300, 512, ["matmul_mx4_tile128"]), ([100] * 40, 1100, 992, ["matmul_mx4_tile128"]),
                                  ([250, 0, 300, 17, 1, 400] * 12, 2048, 1056, ["matmul_mx4_tile256"]), ([130, 0, 257, 300, 5] * 8, 2048, 7168, ["matmul_mx4_tile256"]),
                                  ([64, 0, 100, 1] * 10, 2048, 7168, ["matmul_mx4_tile128"]), ([150, 200] * 300, 512, 544, ["matmul_mx4_tile256"]),
                                  ([1024], 18432, 1024, ["matmul_mx4_tile128"]), ([4] * 240, 900, 1184, ["matmul_mx4_ring"]), ([5, 0, 2], 640, 6016, ["matmul_mx4_stream"]),
                                  ([64], 18432, 1024, ["matmul_mx4_tile128"]), ([64], 640, 1024, ["matmul_mx4_stream"])):
            xc = torch.zeros((sum(sizes), K // 2), dtype=torch.uint8, device="cuda")
            xs = torch.zeros((sum(sizes), moe.mx4_scale_cols(K)), dtype=torch.uint8, device="cuda")
            wc = torch.zeros((len(sizes), N, K // 2), dtype=torch.uint8, device="cuda")
            ws = torch.zeros((len(sizes), N, moe.mx4_scale_cols(K)), dtype=torch.uint8, device="cuda")
            moe.moe_profile_events(events, 8)
            moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes))
            torch.cuda.synchronize()
            got = [moe.moe_profile_kernel(i) for i in range(moe.moe_profile_count())]
            assert got == want, (sizes[:3], N, K, got)
    finally:
        moe.moe_profile_events(None, 0)


@pytest.mark.parametrize("sizes,N,K", [([9, 1, 4] * 60, 700, 1056), ([6111], 5103, 6176), ([300] * 50, 1300, 544), ([250, 0, 300, 17, 1, 400] * 12, 2048, 1056), ([5, 0, 2], 640, 6016)],
                         ids=["ring", "packed", "tile128", "tile256", "stream"])
def test_nan_stays_in_its_row_and_column_on_every_kernel(sizes, N, K):
    """NaN and padding of 255 in the scales; the other results keep their bits."""
    torch = _torch()
    rows, G, blocks = sum(sizes), len(sizes), K // 32
    xc, xs = moe.moe_quantize_mx4(torch.randn((rows, K), device="cuda"))
    wc, ws = _weights(G, N, K, 8)
    want = moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes))
    xs[:, blocks:], ws[:, :, blocks:] = 255, 255
    assert torch.equal(moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes)), want)
    last = max(g for g in range(G) if sizes[g])
    xs[rows - 1, blocks - 1] = 255
    ws[last, N - 3, blocks // 2] = 255
    y = moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes))
    assert bool(y[rows - 1].isnan().all()) and bool(y[rows - sizes[last]:, N - 3].isnan().all())
    want[rows - 1] = float("nan")
    want[rows - sizes[last]:, N - 3] = float("nan")
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.nan_to_num(), want.nan_to_num())


def test_past_four_gib():
    """Weights, rows and results beyond 4 GiB: the last parts are those of small calls."""
    torch = _torch()
    K = 4096
    # 700 groups, 4.9 GB of codes; the last groups' rows
    sizes = [1] * 700
    xc, xs = moe.moe_quantize_mx4(torch.randn((700, K), device="cuda"))
    wc, ws = _weights(700, 3400, K, 1)
    assert wc.numel() > 1 << 32
    y = moe.moe_matmul_mx4(xc, xs, wc, ws, _offsets(sizes))
    part = moe.moe_matmul_mx4(xc[-2:], xs[-2:], wc[-2:], ws[-2:], _offsets([1, 1]), y_dtype=moe.MOE_F32)
    assert bool(((y[-2:].double() - part.double()).abs() <= 2.0 ** -8 * part.double().abs() + 2.0 ** -18 * part.double().abs().max()).all())
    del wc, ws, y
    # 300000 rows of 32768 values: 4.9 GB of codes, 39 GB of bf16
    x = torch.zeros((300000, 32768), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, 32768), device="cuda").bfloat16()
    codes, scales = moe.moe_quantize_mx4(x)
    c, s = moe.moe_quantize_mx4(x[-3:])
    assert torch.equal(codes[-3:], c) and torch.equal(scales[-3:], s) and not bool(codes[:-3].any())
    back = moe.moe_dequantize_mx4(codes, scales, out=x)
    assert torch.equal(back[-3:], moe.moe_dequantize_mx4(c, s)) and not bool(back[:-3].any())
    del x, back
    wc, ws = _weights(1, 70, 32768, 3)
    y = moe.moe_matmul_mx4(codes, scales, wc, ws, y_dtype=moe.MOE_F32)
    part = moe.moe_matmul_mx4(c, s, wc, ws, y_dtype=moe.MOE_F32)
    assert not bool(y[:-3].any()) and bool(((y[-3:] - part).abs() <= 2.0 ** -14 * part.abs().max()).all())
    del codes, scales, y
    # results of 5.6 GB
    xc, xs = moe.moe_quantize_mx4(torch.randn((80000, 64), device="cuda"))
    wc, ws = _weights(1, 17500, 64, 4)
    y = moe.moe_matmul_mx4(xc, xs, wc, ws, y_dtype=moe.MOE_F32)
    part = moe.moe_matmul_mx4(xc[-100:], xs[-100:], wc, ws, y_dtype=moe.MOE_F32)
    assert bool(((y[-100:] - part).abs() <= 2.0 ** -20 * part.abs().max()).all())
