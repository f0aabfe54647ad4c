"""Grouped matrix products, their gradients and the 8-bit integer products (include/moe.h) against
float64 evaluations of their formulas.

Bounds, per output element, derived from the arithmetic:
* fp32 sums of `depth` products: (depth + 16) 2^-23 sum |a b| (every addition rounds once; the products
  of bf16 values are exact, those of fp32 values round inside the fused multiply-add);
* the output's rounding: 2^-8 |y| for bf16 (half a step of 7 fraction bits), 2^-23 |y| for fp32;
* 8-bit integers: the int32 sum is exact; its conversion to fp32 and two scale products round three times,
  3 * 2^-24 |y|, plus the output's rounding.
"""
import numpy as np
import pytest

import moe_layer_forward_amd as moe

pytestmark = pytest.mark.gpu


def _torch():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _dt(name):
    torch = _torch()
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _np(t):
    return t.detach().double().cpu().numpy()


def _offsets(G, rows, spread, seed):
    """[G + 1] group offsets: even (multinomial), skew (two groups take most rows, many are empty), last
    (every row in the last group), first (every row in the first group)."""
    rng = np.random.default_rng(seed)
    if spread == "even":
        n = rng.multinomial(rows, np.ones(G) / G)
    elif spread == "skew":
        p = np.zeros(G)
        p[rng.permutation(G)[:max(1, G // 3)]] = 1.0
        p[rng.integers(G)] += 4.0
        n = rng.multinomial(rows, p / p.sum())
    else:
        n = np.zeros(G, np.int64)
        n[0 if spread == "first" else G - 1] = rows
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def _dev(a, dt=None):
    torch = _torch()
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dt is None else t.to(dt)


def _check(got, ref, absum, depth, out_dtype, what):
    out = 2.0 ** -8 if out_dtype == "bf16" else 2.0 ** -23
    bound = out * np.abs(ref) + (depth + 16) * 2.0 ** -23 * absum + 1e-37
    err = np.abs(_np(got) - ref)
    worst = float((err / bound).max()) if err.size else 0.0
    assert np.all(err <= bound), f"{what}: {worst:.3g} times the bound"
    print(f"{what}: at most {worst:.3g} of the bound", flush=True)


def _groups(off):
    return [slice(int(off[g]), int(off[g + 1])) for g in range(len(off) - 1)]


# (G, rows, N, K, spread): every size from one on; row lengths that are and are not multiples of 16 bytes;
# tiles that end inside, at and past 16, 64, 128 and 256; more groups than lanes; empty groups
SIZES = [
    (1, 1, 1, 1, "even"), (1, 5, 3, 7, "even"), (1, 1, 8, 16, "even"), (2, 3, 17, 33, "last"),
    (16, 128, 128, 256, "even"), (4, 100, 130, 70, "skew"), (5, 300, 257, 191, "skew"), (3, 257, 128, 64, "first"),
    (7, 129, 40, 1000, "even"), (70, 500, 64, 72, "even"), (130, 200, 96, 128, "skew"), (2, 1000, 511, 513, "even"),
    (3, 640, 512, 384, "even"), (4, 900, 264, 136, "skew"), (9, 31, 320, 448, "even"), (1, 700, 1032, 2056, "even"),
    (6, 1500, 72, 520, "skew"), (24, 48, 1024, 768, "even"),
]
IDS = ["G%d_R%d_N%d_K%d_%s" % s for s in SIZES]


def _case(size, dt, gather, seed=0):
    G, rows, N, K, spread = size
    torch = _torch()
    off = _offsets(G, rows, spread, seed + 1)
    rng = np.random.default_rng(seed)
    x_rows = max(1, rows // 3) if gather else rows
    idx = rng.integers(0, x_rows, rows) if gather else np.arange(rows)
    x = _dev(rng.standard_normal((x_rows, K)), _dt(dt))
    w = _dev(rng.standard_normal((G, N, K)) / np.sqrt(K), _dt(dt))
    dy = _dev(rng.standard_normal((rows, N)), _dt(dt))
    d_idx = _dev(idx.astype(np.int32)) if gather else None
    d_off = _dev(off.astype(np.int32))
    torch.cuda.synchronize()
    return off, idx, x, w, dy, d_off, d_idx


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_forward(size, dt, gather):
    off, idx, x, w, _, d_off, d_idx = _case(size, dt, gather)
    G, rows, N, K, _ = size
    torch = _torch()
    out_dt = "f32" if dt == "f32" or size[0] % 2 else "bf16"
    y = torch.full((rows, N), float("nan"), dtype=_dt(out_dt), device="cuda")
    moe.moe_grouped_matmul(x, w, d_off, row_index=d_idx, out=y)
    xn, wn = _np(x)[idx], _np(w)
    ref, ab = np.zeros((rows, N)), np.zeros((rows, N))
    for g, r in enumerate(_groups(off)):
        ref[r], ab[r] = xn[r] @ wn[g].T, np.abs(xn[r]) @ np.abs(wn[g]).T
    _check(y, ref, ab, K, out_dt, "y")
    # the default output has the inputs' type
    y2 = moe.moe_grouped_matmul(x, w, d_off, row_index=d_idx)
    assert y2.dtype == x.dtype and torch.equal(y2, y.to(x.dtype) if out_dt == "f32" else y)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_gradient_for_rows(size, dt):
    off, _, _, w, dy, d_off, _ = _case(size, dt, False, seed=3)
    G, rows, N, K, _ = size
    torch = _torch()
    out_dt = "f32" if dt == "f32" or size[0] % 2 else "bf16"
    dx = torch.full((rows, K), float("nan"), dtype=_dt(out_dt), device="cuda")
    moe.moe_grouped_matmul_dx(dy, w, d_off, out=dx)
    dn, wn = _np(dy), _np(w)
    ref, ab = np.zeros((rows, K)), np.zeros((rows, K))
    for g, r in enumerate(_groups(off)):
        ref[r], ab[r] = dn[r] @ wn[g], np.abs(dn[r]) @ np.abs(wn[g])
    _check(dx, ref, ab, N, out_dt, "dx")


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_gradient_for_weights(size, dt, gather):
    off, idx, x, _, dy, d_off, d_idx = _case(size, dt, gather, seed=5)
    G, rows, N, K, _ = size
    torch = _torch()
    out_dt = "f32" if dt == "f32" or size[0] % 2 else "bf16"
    dw = torch.full((G, N, K), float("nan"), dtype=_dt(out_dt), device="cuda")
    moe.moe_grouped_matmul_dw(dy, x, d_off, row_index=d_idx, out=dw)
    xn, dn = _np(x)[idx], _np(dy)
    ref, ab = np.zeros((G, N, K)), np.zeros((G, N, K))
    for g, r in enumerate(_groups(off)):
        ref[g], ab[g] = dn[r].T @ xn[r], np.abs(dn[r]).T @ np.abs(xn[r])
    _check(dw, ref, ab, int(max(np.diff(off).max(), 1)), out_dt, "dw")
    for g in range(G):
        if off[g] == off[g + 1]:
            assert bool((dw[g] == 0).all()), f"empty group {g} has a gradient"


# few output tiles and long sums: groups whose rows are cut into ranges, beside groups that are one range or none
LONG_SUMS = [(1, 5000, 64, 64, "even"), (2, 4099, 200, 136, "even"), (5, 2500, 200, 136, "skew"),
             (9, 4100, 65, 67, "skew"), (40, 3000, 96, 72, "first"), (40, 3001, 96, 72, "last"),
             (300, 6000, 128, 264, "skew"), (7, 9000, 520, 8, "skew")]


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", LONG_SUMS, ids=["-".join(map(str, s)) for s in LONG_SUMS])
def test_gradient_for_weights_of_long_groups(size, dt, gather):
    test_gradient_for_weights(size, dt, gather)
    off, idx, x, _, dy, d_off, d_idx = _case(size, dt, gather, seed=6)
    dw = moe.moe_grouped_matmul_dw(dy, x, d_off, row_index=d_idx)
    assert _torch().equal(dw, moe.moe_grouped_matmul_dw(dy, x, d_off, row_index=d_idx))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_one_group_without_offsets(dt):
    torch = _torch()
    off, idx, x, w, dy, d_off, _ = _case((1, 300, 200, 328, "even"), dt, False, seed=8)
    assert torch.equal(moe.moe_grouped_matmul(x, w, None), moe.moe_grouped_matmul(x, w, d_off))
    assert torch.equal(moe.moe_grouped_matmul_dx(dy, w, None), moe.moe_grouped_matmul_dx(dy, w, d_off))
    assert torch.equal(moe.moe_grouped_matmul_dw(dy, x, None), moe.moe_grouped_matmul_dw(dy, x, d_off))


def test_no_rows():
    """No rows: nothing to write for the rows, zeros for the weights' gradient."""
    torch = _torch()
    x = torch.empty((0, 48), dtype=torch.bfloat16, device="cuda")
    dy = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((3, 40, 48), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert moe.moe_grouped_matmul(x, w, off).shape == (0, 40)
    assert moe.moe_grouped_matmul_dx(dy, w, off).shape == (0, 48)
    dw = torch.full((3, 40, 48), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_matmul_dw(dy, x, off, out=dw)
    assert bool((dw == 0).all())
    q, s = moe.moe_quantize_rows(x)
    assert q.shape == (0, 48) and s.shape == (0,)


@pytest.mark.parametrize("K,N", [(128, 256), (100, 72), (33, 35)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_past_the_last_group_are_not_written(dt, K, N):
    torch = _torch()
    off = torch.tensor([0, 40, 40, 90], dtype=torch.int32, device="cuda")
    x = torch.randn((150, K), device="cuda").to(_dt(dt))
    dy = torch.randn((150, N), device="cuda").to(_dt(dt))
    x[90:], dy[90:] = float("nan"), float("nan")
    w = torch.randn((3, N, K), device="cuda").to(_dt(dt))
    y = torch.full((150, N), 7.0, dtype=_dt(dt), device="cuda")
    dx = torch.full((150, K), 7.0, dtype=_dt(dt), device="cuda")
    moe.moe_grouped_matmul(x, w, off, out=y)
    moe.moe_grouped_matmul_dx(dy, w, off, out=dx)
    dw = moe.moe_grouped_matmul_dw(dy, x, off)
    assert bool((y[90:] == 7.0).all()) and bool((dx[90:] == 7.0).all())
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())
    # fewer rows than the bound may run on another kernel or split: within two roundings of the sums
    for a, b in ((y[:90], moe.moe_grouped_matmul(x[:90].contiguous(), w, off)),
                 (dw, moe.moe_grouped_matmul_dw(dy[:90].contiguous(), x[:90].contiguous(), off))):
        assert bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs() + 2e-3).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("N,K", [(128, 192), (264, 520), (70, 45)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_non_finite_values_stay_in_their_row_and_group(dt, N, K, bad):
    """One bad row of group 1 and one bad weight of group 2 touch exactly the outputs that sum over them."""
    torch = _torch()
    off = [0, 50, 83, 83, 300]
    d_off = torch.tensor(off, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    x = torch.rand((300, K), device="cuda", generator=gen).add_(0.5).to(_dt(dt))
    dy = torch.rand((300, N), device="cuda", generator=gen).add_(0.5).to(_dt(dt))
    w = torch.rand((4, N, K), device="cuda", generator=gen).add_(0.5).to(_dt(dt))
    x[60, K - 1], dy[60, N - 1], w[3, N - 1, K - 1] = bad, bad, bad
    y = moe.moe_grouped_matmul(x, w, d_off)
    dx = moe.moe_grouped_matmul_dx(dy, w, d_off)
    dw = moe.moe_grouped_matmul_dw(dy, x, d_off)
    hit = torch.zeros((300, N), dtype=torch.bool, device="cuda")
    hit[60] = True
    hit[83:, N - 1] = True
    assert torch.equal(~torch.isfinite(y), hit)
    hit = torch.zeros((300, K), dtype=torch.bool, device="cuda")
    hit[60] = True
    hit[83:, K - 1] = True
    assert torch.equal(~torch.isfinite(dx), hit)
    hit = torch.zeros((4, N, K), dtype=torch.bool, device="cuda")
    hit[1, N - 1] = True
    hit[1, :, K - 1] = True
    assert torch.equal(~torch.isfinite(dw), hit)


@pytest.mark.parametrize("size", [(3, 120, 72, 56, "even"), (5, 600, 264, 136, "skew")])
def test_gradients_against_differences(size):
    """The product is linear in the rows and in the weights, so central differences of fp32 forwards have no
    truncation error: <dy, y(x + d) - y(x - d)> / 2 = <dx, d>, and likewise for the weights.  Both sides are
    sums of R N K fp32 products: the bound is their rounding, (depth + 16) 2^-23 of the absolute sums."""
    off, idx, x, w, dy, d_off, d_idx = _case(size, "f32", True, seed=9)
    torch = _torch()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    xr = x[d_idx.long()].contiguous()
    d = torch.randn(xr.shape, generator=gen, device="cuda")
    e = torch.randn(w.shape, generator=gen, device="cuda")
    plus, minus = (moe.moe_grouped_matmul(xr + s * d, w, d_off).double() for s in (1, -1))
    dx = moe.moe_grouped_matmul_dx(dy, w, d_off).double()
    lhs, rhs = ((plus - minus) / 2 * dy.double()).sum(), (dx * d.double()).sum()
    big = max(size[2], size[3]) + 16
    ab = sum(float((dy[r].abs().double() @ w[g].abs().double() * (xr[r].abs() + d[r].abs()).double()).sum())
             for g, r in enumerate(_groups(off)))
    assert abs(float(lhs - rhs)) <= 3 * big * 2.0 ** -23 * ab
    plus, minus = (moe.moe_grouped_matmul(x, w + s * e, d_off, row_index=d_idx).double() for s in (1, -1))
    dw = moe.moe_grouped_matmul_dw(dy, x, d_off, row_index=d_idx).double()
    lhs, rhs = ((plus - minus) / 2 * dy.double()).sum(), (dw * e.double()).sum()
    ab = sum(float((dy[r].abs().double().T @ xr[r].abs().double() * (w[g].abs() + e[g].abs()).double()).sum())
             for g, r in enumerate(_groups(off)))
    assert abs(float(lhs - rhs)) <= 3 * (size[1] + big) * 2.0 ** -23 * ab


def test_gathered_rows_gradient_per_token():
    """A token's gradient is the sum over its rows: moe_combine with weights 1 adds the rows' dx."""
    torch = _torch()
    T, K2, E, N, K = 90, 4, 12, 192, 256
    cfg = moe.make_config(hidden_size=K, moe_intermediate_size=128, n_routed_experts=E, top_k=K2, n_shared_experts=0,
                          dtype="f32")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    ids = torch.stack([torch.randperm(E, generator=gen, device="cuda")[:K2] for _ in range(T)]).int().contiguous()
    off, row_token, pair_row, _ = moe.moe_permute(cfg, ids)
    w = torch.randn((E, N, K), generator=gen, device="cuda")
    dy = torch.randn((T * K2, N), generator=gen, device="cuda")
    dx = moe.moe_grouped_matmul_dx(dy, w, off)
    got = moe.moe_combine(cfg, dx, pair_row, torch.ones((T, K2), device="cuda"))
    o = off.cpu().numpy()
    dn, wn, tok = _np(dy), _np(w), row_token.cpu().numpy()
    ref, ab = np.zeros((T, K)), np.zeros((T, K))
    for g, r in enumerate(_groups(o)):
        np.add.at(ref, tok[r], dn[r] @ wn[g])
        np.add.at(ab, tok[r], np.abs(dn[r]) @ np.abs(wn[g]))
    _check(got, ref, ab, N + K2, "f32", "dx per token")


def test_unaligned_starts():
    """Operands that start on any element boundary (slices of larger buffers)."""
    torch = _torch()
    off, _, x, w, dy, d_off, _ = _case((3, 200, 128, 256, "even"), "bf16", False, seed=12)

    def moved(t):
        big = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        big[1:] = t.reshape(-1)
        return big[1:].view(t.shape)

    for a, b in ((moe.moe_grouped_matmul(x, w, d_off), moe.moe_grouped_matmul(moved(x), moved(w), d_off)),
                 (moe.moe_grouped_matmul_dx(dy, w, d_off), moe.moe_grouped_matmul_dx(moved(dy), moved(w), d_off)),
                 (moe.moe_grouped_matmul_dw(dy, x, d_off), moe.moe_grouped_matmul_dw(moved(dy), moved(x), d_off))):
        # other kernels may add in another order: at most one bf16 step apart
        assert bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs() + 1e-3).all())
    y = moved(torch.zeros((200, 128), dtype=torch.bfloat16, device="cuda"))
    moe.moe_grouped_matmul(x, w, d_off, out=y)
    assert torch.equal(y, moe.moe_grouped_matmul(x, w, d_off))


def test_outside_row_index_reads_inside():
    """Indices outside x are moved inside: no fault, and the other rows keep their results."""
    torch = _torch()
    for K in (128, 50):
        x = torch.randn((64, K), device="cuda").bfloat16()
        w = torch.randn((2, 96, K), device="cuda").bfloat16()
        off = torch.tensor([0, 30, 100], dtype=torch.int32, device="cuda")
        good = torch.randint(0, 64, (100,), device="cuda", dtype=torch.int32)
        bad = good.clone()
        bad[5], bad[77] = -3, 2 ** 31 - 1
        a, b = (moe.moe_grouped_matmul(x, w, off, row_index=i) for i in (good, bad))
        keep = torch.ones(100, dtype=torch.bool, device="cuda")
        keep[5] = keep[77] = False
        assert torch.equal(a[keep], b[keep])
        dy = torch.randn((100, 96), device="cuda").bfloat16()
        assert bool(torch.isfinite(moe.moe_grouped_matmul_dw(dy, x, off, row_index=bad)).all())


@pytest.mark.parametrize("long", ["rows_in", "rows_out"])
def test_offsets_past_32_bits(long):
    """Row operands and outputs of more than 4 GiB: the last rows against the formula."""
    torch = _torch()
    rows = 700_001
    N, K = (16, 4096) if long == "rows_in" else (4096, 16)
    off = torch.tensor([0, 300_000, 300_100, rows], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x = torch.randn((rows, K), generator=gen, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn((rows, N), generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.randn((3, N, K), generator=gen, device="cuda", dtype=torch.bfloat16)
    y = moe.moe_grouped_matmul(x, w, off)
    dx = moe.moe_grouped_matmul_dx(dy, w, off)
    dw = moe.moe_grouped_matmul_dw(dy, x, off, dw_dtype=moe.MOE_F32)
    for r, g in ((slice(0, 50), 0), (slice(300_000, 300_100), 1), (slice(rows - 60, rows), 2)):
        xs, ds, ws = x[r].double(), dy[r].double(), w[g].double()
        for got, ref, ab, depth in ((y[r], xs @ ws.T, xs.abs() @ ws.abs().T, K),
                                    (dx[r], ds @ ws, ds.abs() @ ws.abs(), N)):
            _check(got, _np(ref), _np(ab), depth, "bf16", f"rows {r}")
    for g in range(3):
        r = slice(int(off[g]), int(off[g + 1]))
        ref = sum(dy[i:i + 50_000].double().T @ x[i:min(i + 50_000, r.stop)].double() if i + 50_000 <= r.stop else
                  dy[i:r.stop].double().T @ x[i:r.stop].double() for i in range(r.start, r.stop, 50_000))
        n = r.stop - r.start
        # sums of n products of normals: |dy x| sums to about 0.64 n, at most n for these lengths
        err = (dw[g].double() - ref).abs()
        assert bool((err <= (n + 16) * 2.0 ** -23 * n).all()), f"dw of group {g}"


# --------------------------------------------------------------------------- 8-bit integers
def _quant_ref(v):
    a = np.abs(v).max(axis=1)
    q = np.rint(127.0 * v / np.where(a > 0, a, 1.0)[:, None])
    return q, a / 127.0


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 64), (17, 333), (64, 2048), (9, 2056), (33, 7168),
                                       (2, 16384), (3, 20011), (4, 40000)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_rows(rows, cols, dt):
    """bf16: the codes of the formula, exactly.  fp32: 127 v and the quotient round to 24 bits, so a code may
    differ where the exact quotient is within 127 * 2^-22 of a tie."""
    torch = _torch()
    rng = np.random.default_rng(rows * 1000 + cols)
    x = _dev(rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-20, 20, (rows, 1))), _dt(dt))
    x[0, cols // 2] = x[0].abs().max() / 2 if cols > 1 else x[0, 0]  # half the maximum: the quotient 63.5, a tie
    codes = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda")
    codes, scales = moe.moe_quantize_rows(x, codes=codes)
    xn = _np(x)
    q, s = _quant_ref(xn)
    got = _np(codes)
    if dt == "bf16":
        assert np.array_equal(got, q)
    else:
        exact = 127.0 * xn / np.abs(xn).max(axis=1)[:, None]
        tie = np.abs(np.abs(exact - np.floor(exact)) - 0.5) <= 127 * 2.0 ** -22
        assert np.all((got == q) | (tie & (np.abs(got - q) <= 1)))
    assert np.all(np.abs(_np(scales) - s) <= 2.0 ** -24 * s)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_special_rows(dt):
    torch = _torch()
    for cols in (40, 5000):
        x = torch.ones((8, cols), device="cuda")
        x[0] = 0
        x[1, 3] = float("nan")
        x[2, cols - 1] = float("-inf")
        x[3] = 3e38
        x[3, 0] = -3e38
        x[4] = 1e-39
        x[5] = -0.0
        x[6, 0] = 2.0
        x = x.to(_dt(dt))
        codes, scales = moe.moe_quantize_rows(x)
        c, s = codes.cpu().numpy(), scales.cpu().numpy()
        assert np.all(c[0] == 0) and s[0] == 0 and np.all(c[5] == 0) and s[5] == 0
        assert np.isnan(s[1]) and np.isnan(s[2]) and np.all(c[1:3] == 0)
        assert np.all(c[3, 1:] == 127) and c[3, 0] == -127 and abs(s[3] / (3e38 / 127) - 1) < 0.01
        assert np.all(c[4] == 127)
        assert c[6, 0] == 127 and np.all(c[6, 1:] == 64)  # 63.5 goes to the even 64
        assert np.all(c[7] == 127)


@pytest.mark.parametrize("rows,cols", [(1, 1), (4, 30), (40, 2048), (7, 2500), (3, 18000)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_swiglu(rows, cols, dt):
    """SiLU(gate) * up in fp32 (exp, one division, two products: within 2^-20 relative), then the codes:
    within one of the formula's, and equal wherever its quotient is 127 * 2^-18 or more from a tie."""
    rng = np.random.default_rng(rows + cols)
    x = _dev(rng.standard_normal((rows, 2 * cols)) * 3, _dt(dt))
    codes, scales = moe.moe_quantize_rows(x, swiglu=True)
    xn = _np(x)
    g, u = xn[:, :cols], xn[:, cols:]
    v = g / (1 + np.exp(-g)) * u
    q, s = _quant_ref(v)
    exact = 127.0 * v / np.abs(v).max(axis=1)[:, None]
    tie = np.abs(np.abs(exact - np.floor(exact)) - 0.5) <= 127 * 2.0 ** -18
    got = _np(codes)
    assert codes.shape == (rows, cols)
    assert np.all((got == q) | (tie & (np.abs(got - q) <= 1)))
    assert np.all(np.abs(_np(scales) - s) <= 2.0 ** -19 * s)


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
@pytest.mark.parametrize("out_dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_matmul_i8(size, out_dt, gather):
    G, rows, N, K, spread = size
    torch = _torch()
    rng = np.random.default_rng(21)
    off = _offsets(G, rows, spread, 22)
    x_rows = max(1, rows // 3) if gather else rows
    idx = rng.integers(0, x_rows, rows) if gather else np.arange(rows)
    xc = rng.integers(-128, 128, (x_rows, K)).astype(np.int8)
    wc = rng.integers(-128, 128, (G, N, K)).astype(np.int8)
    xs = rng.uniform(0.5, 2, x_rows).astype(np.float32)
    ws = rng.uniform(0.5, 2, (G, N)).astype(np.float32)
    y = torch.full((rows, N), float("nan"), dtype=_dt(out_dt), device="cuda")
    moe.moe_matmul_i8(_dev(xc), _dev(xs), _dev(wc), _dev(ws), _dev(off.astype(np.int32)),
                      row_index=_dev(idx.astype(np.int32)) if gather else None, out=y)
    ref = np.zeros((rows, N))
    for g, r in enumerate(_groups(off)):
        ref[r] = (xc[idx[r]].astype(np.float64) @ wc[g].astype(np.float64).T) * xs[idx[r]][:, None] * ws[g]
    bound = (3 * 2.0 ** -24 + (2.0 ** -8 if out_dt == "bf16" else 0.0)) * np.abs(ref) * 1.0001
    err = np.abs(_np(y) - ref)
    assert np.all(err <= bound), float((err - bound).max())


def test_matmul_i8_extremes():
    """The longest contraction with every code at -128: the sum stays inside int32."""
    torch = _torch()
    K = 131071
    x = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((1, 5, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(5, device="cuda")
    y = moe.moe_matmul_i8(x, one[:3].contiguous(), w, one.view(1, 5), y_dtype=moe.MOE_F32)
    assert bool((y == float(np.float32(K * 16384))).all())
    s = torch.tensor([1.0, float("nan"), 0.0], device="cuda")  # a row that could not be quantized, a zero row
    y = moe.moe_matmul_i8(x, s, w, one.view(1, 5))
    assert bool(torch.isnan(y[1]).all()) and bool((y[2] == 0).all()) and bool(torch.isfinite(y[0]).all())


@pytest.mark.parametrize("T,E,H,I", [(40, 6, 256, 192), (130, 4, 200, 72)])
def test_int8_expert_ffn_follows_the_float_one(T, E, H, I):
    """Quantize, gate and up, SwiGLU and quantize, down against the same steps in float64 with the codes' exact
    rounding: codes of the intermediate may differ by one where its quotient is near a tie, which moves an
    output by at most one step of one term, scale_h * |w|: allowed for 1% of the terms."""
    torch = _torch()
    rng = np.random.default_rng(5)
    off = _offsets(E, T, "even", 6)
    x = _dev(rng.standard_normal((T, H)), torch.bfloat16)
    wc, dc = (rng.integers(-127, 128, s).astype(np.int8) for s in ((E, 2 * I, H), (E, H, I)))
    ws = (rng.uniform(0.8, 1.2, (E, 2 * I)) / 73 / np.sqrt(H)).astype(np.float32)
    ds = (rng.uniform(0.8, 1.2, (E, H)) / 73 / np.sqrt(I)).astype(np.float32)
    d_off = _dev(off.astype(np.int32))
    q, s = moe.moe_quantize_rows(x)
    gu = moe.moe_matmul_i8(q, s, _dev(wc), _dev(ws), d_off, y_dtype=moe.MOE_F32)
    h, sh = moe.moe_quantize_rows(gu, swiglu=True)
    y = _np(moe.moe_matmul_i8(h, sh, _dev(dc), _dev(ds), d_off, y_dtype=moe.MOE_F32))
    qr, sr = _quant_ref(_np(x))
    for g, r in enumerate(_groups(off)):
        if r.start == r.stop:
            continue
        a = (qr[r] @ wc[g].astype(np.float64).T) * sr[r][:, None] * ws[g]
        v = a[:, :I] / (1 + np.exp(-a[:, :I])) * a[:, I:]
        hq, hs = _quant_ref(v)
        ref = (hq @ dc[g].astype(np.float64).T) * hs[:, None] * ds[g]
        step = hs[:, None] * ds[g] * 127
        assert np.all(np.abs(y[r] - ref) <= max(1.0, 0.01 * I) * step + 2.0 ** -18 * np.abs(ref))
        assert np.mean(np.abs(y[r] - ref) > 2.0 ** -18 * np.abs(ref) + 1e-6) < 0.2


# --------------------------------------------------------------------------- how calls behave
def _all_calls(x, w, dy, off, idx, ws=None):
    q, s = moe.moe_quantize_rows(x)
    wq = torch_round(w)
    return [moe.moe_grouped_matmul(x, w, off, row_index=idx), moe.moe_grouped_matmul_dx(dy, w, off),
            moe.moe_grouped_matmul_dw(dy, x, off, row_index=idx), q, s,
            moe.moe_matmul_i8(q, s, wq, w[:, :, 0].float().contiguous(), off, row_index=idx)]


def torch_round(w):
    torch = _torch()
    return (w.float() * 60).clamp(-127, 127).round().to(torch.int8)


@pytest.mark.parametrize("size", [(4, 500, 256, 320, "skew"), (3, 90, 50, 35, "even"), (20, 40, 256, 512, "even"),
                                  (1, 64, 640, 2048, "even")])
def test_calls_repeat_and_run_on_their_stream(size):
    """The same bits on every call, on a stream of the caller's, and with leftover workspace contents."""
    torch = _torch()
    _, _, x, w, dy, off, idx = _case(size, "bf16", True, seed=31)
    first = _all_calls(x, w, dy, off, idx)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            again = _all_calls(x, w, dy, off, idx)
            side.synchronize()
            for a, b in zip(first, again):
                assert torch.equal(a, b)


@pytest.mark.parametrize("size", [(4, 500, 256, 320, "skew"), (20, 40, 256, 512, "even"), (1, 64, 640, 2048, "even"),
                                  (3, 90, 50, 35, "even")])
def test_graph_replays_match_eager(size):
    torch = _torch()
    G, rows, N, K, _ = size
    _, _, x, w, dy, off, idx = _case(size, "bf16", True, seed=33)
    wq, wsc = torch_round(w), w[:, :, 0].float().contiguous()

    def spaces(op, dt):
        n = moe.moe_matmul_workspace_size(op, dt, G, rows, N, K)
        return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")

    wss = [spaces(op, moe.MOE_BF16) for op in range(4)]
    y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    y8 = torch.empty_like(y)
    dx = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((G, N, K), dtype=torch.bfloat16, device="cuda")
    q = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    s = torch.empty(x.shape[0], device="cuda")

    def call():
        moe.moe_grouped_matmul(x, w, off, row_index=idx, out=y, workspace=wss[0])
        moe.moe_grouped_matmul_dx(dy, w, off, out=dx, workspace=wss[1])
        moe.moe_grouped_matmul_dw(dy, x, off, row_index=idx, out=dw, workspace=wss[2])
        moe.moe_quantize_rows(x, codes=q, scales=s)
        moe.moe_matmul_i8(q, s, wq, wsc, off, row_index=idx, out=y8, workspace=wss[3])

    outs = (y, dx, dw, q, s, y8)
    inputs = [x.clone(), torch.flip(x, dims=[0]).contiguous()]
    refs = []
    for xin in inputs:
        x.copy_(xin)
        call()
        torch.cuda.synchronize()
        refs.append([o.clone() for o in outs])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    torch.cuda.synchronize()
    for rep in range(4):
        x.copy_(inputs[rep % 2])
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, refs[rep % 2]):
            assert torch.equal(o, r), f"replay {rep}"


def test_refusals_on_the_device():
    """Wrong types, shapes and layouts raise before anything runs; outputs keep their contents."""
    torch = _torch()
    x = torch.zeros((10, 32), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 24, 32), dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros((10, 24), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 4, 10], dtype=torch.int32, device="cuda")
    for bad in (lambda: moe.moe_grouped_matmul(x.half(), w, off),
                lambda: moe.moe_grouped_matmul(x, w.float(), off),
                lambda: moe.moe_grouped_matmul(x[:, :31].contiguous(), w, off),
                lambda: moe.moe_grouped_matmul(x[:, ::2], w[:, :, :16].contiguous(), off),
                lambda: moe.moe_grouped_matmul(x, w, off.long()),
                lambda: moe.moe_grouped_matmul(x, w, off[:2].contiguous()),
                lambda: moe.moe_grouped_matmul(x, w, None),
                lambda: moe.moe_grouped_matmul(x, w, off, row_index=torch.zeros(10, device="cuda")),
                lambda: moe.moe_grouped_matmul(x, w, off, out=torch.zeros((10, 23), device="cuda")),
                lambda: moe.moe_grouped_matmul(x, w, off, y_dtype=9),
                lambda: moe.moe_grouped_matmul(x.cpu(), w, off),
                lambda: moe.moe_grouped_matmul_dx(dy[:, :20].contiguous(), w, off),
                lambda: moe.moe_grouped_matmul_dw(dy, x[:9].contiguous(), off),
                lambda: moe.moe_grouped_matmul_dw(dy, x.float(), off),
                lambda: moe.moe_quantize_rows(x.half()),
                lambda: moe.moe_quantize_rows(x[:, :31].contiguous(), swiglu=True),
                lambda: moe.moe_quantize_rows(x, codes=torch.zeros((10, 32), device="cuda")),
                lambda: moe.moe_matmul_i8(x, off.float(), w, off.float(), off)):
        with pytest.raises(ValueError):
            bad()
