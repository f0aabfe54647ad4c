"""The grouped products on each of their kernels: what a call launched is read from the library's own
profile (moe_profile_events), so that a test which is about one kernel fails where another runs."""
import ctypes

import numpy as np
import pytest

import moe_layer_forward_amd as moe

pytestmark = pytest.mark.gpu


def _torch():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _launched(call, n_events=16):
    """(what call returns, [(kernel, ms)] of what it launched)."""
    torch = _torch()
    events = [torch.cuda.Event(enable_timing=True) for _ in range(n_events)]
    for e in events:
        e.record()  # torch creates an event when it is first recorded
    handles = (ctypes.c_void_p * n_events)(*[e.cuda_event for e in events])
    torch.cuda.synchronize()
    moe.moe_profile_events(handles, n_events)
    try:
        out = call()
        n = moe.moe_profile_count()
        names = [moe.moe_profile_kernel(i) for i in range(n)]
    finally:
        moe.moe_profile_events(None, 0)
    torch.cuda.synchronize()
    return out, [(k, events[2 * i].elapsed_time(events[2 * i + 1])) for i, k in enumerate(names)]


def test_profile_has_one_entry_per_launch():
    """A call whose sums are split launches the product and the join, and each is timed by itself."""
    torch = _torch()
    x = torch.randn((64, 8192), device="cuda").bfloat16()
    w = torch.randn((1, 128, 8192), device="cuda").bfloat16()
    dy = torch.randn((64, 128), device="cuda").bfloat16()
    rows = torch.randn((5000, 64), device="cuda")
    q, s = moe.moe_quantize_rows(x)
    qw, sw = moe.moe_quantize_rows(w[0])
    for call, want in (
            (lambda: moe.moe_grouped_matmul(x, w, None), ["matmul_tile128", "matmul_join"]),
            (lambda: moe.moe_grouped_matmul(x.float(), w.float(), None), ["matmul_any64", "matmul_join"]),
            (lambda: moe.moe_matmul_i8(q, s, qw[None], sw[None]), ["matmul_tile128", "matmul_join"]),
            (lambda: moe.moe_grouped_matmul_dw(rows, rows, None), ["matmul_any64", "matmul_join"]),
            (lambda: moe.moe_grouped_matmul_dx(dy, w, None), ["matmul_tile128"]),
            (lambda: moe.moe_quantize_rows(x), ["quantize_rows"])):
        _, got = _launched(call)
        assert [k for k, _ in got] == want
        assert all(ms > 0 for _, ms in got)


# --------------------------------------------------------------------------- the 256 x 256 and non-temporal kernels
# Small whole numbers: every partial sum is a whole number below 2^24, so that fp32 sums are exact in any
# order and each output has to equal the formula's, rounded once.  A term that is lost, doubled or taken from a
# neighbour (a wait too few, a wrong stage or row) shows by itself.
TOP = 4


def _ints(gen, *shape, top=TOP):
    torch = _torch()
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda", dtype=torch.int8)


def _offsets(sizes):
    torch = _torch()
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return off, torch.from_numpy(off).cuda()


def _exact(a, b, out_dtype, scale=None):
    """a b of whole numbers (float64 holds them), rounded once to out_dtype."""
    torch = _torch()
    y = a.double() @ b.double().contiguous()
    if scale is not None:
        y = y * scale
    return y.float().to(out_dtype) if out_dtype == torch.bfloat16 else y.to(out_dtype)


# a partial tile of 1 to 8 blocks of 32 rows, alone and after a full tile; an empty group between them
ALL_BLOCKS = [20, 256 + 50, 90, 0, 120, 256 + 150, 190, 256 + 220, 250]


def _rows_case(op, sizes, N, K, gather, seed):
    torch = _torch()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    off, d_off = _offsets(sizes)
    rows, G = int(off[-1]), len(sizes)
    depth = N if op == "dx" else K
    x_rows = rows // 3 if gather else rows
    x = _ints(gen, x_rows, depth)
    w = _ints(gen, G, N, K)
    idx = torch.randint(0, x_rows, (rows,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    return off, d_off, x, w, idx


def _check_rows(op, kernel, sizes, N, K, gather, out_name, seed):
    torch = _torch()
    off, d_off, x, w, idx = _rows_case(op, sizes, N, K, gather, seed)
    out_dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[out_name]
    out = torch.full((int(off[-1]), K if op == "dx" else N), float("nan"), dtype=out_dtype, device="cuda")
    xs = ws = None
    if op == "i8":
        # powers of two, so that the scaled values are exact too
        xs = 2.0 ** (torch.arange(x.shape[0], device="cuda") % 5 - 2).float()
        ws = 2.0 ** (torch.arange(len(sizes) * N, device="cuda") % 7 - 3).float().view(len(sizes), N)

        def call():
            return moe.moe_matmul_i8(x, xs, w, ws, d_off, row_index=idx, out=out)
    else:
        xb, wb = x.bfloat16(), w.bfloat16()

        def call():
            if op == "dx":
                return moe.moe_grouped_matmul_dx(xb, wb, d_off, out=out)
            return moe.moe_grouped_matmul(xb, wb, d_off, row_index=idx, out=out)

    _, names = _launched(call)
    assert [k for k, _ in names] == [kernel]
    first = out.clone()
    rows_x = x if idx is None else x[idx.long()]
    for g in range(len(sizes)):
        r = slice(int(off[g]), int(off[g + 1]))
        scale = None
        if op == "i8":
            rs = xs if idx is None else xs[idx.long()]
            scale = rs[r, None].double() * ws[g].double()
        want = _exact(rows_x[r], w[g] if op == "dx" else w[g].T, out_dtype, scale)
        assert torch.equal(first[r], want), f"group {g}: {int((first[r] != want).sum())} values differ"
    for _ in range(3):  # behind one another, over the last results
        call()
    assert torch.equal(out, first)


@pytest.mark.parametrize("steps", range(1, 15))
@pytest.mark.parametrize("op", ["forward", "dx", "i8"])
def test_rows_in_256_tiles(op, steps):
    """Sums of 1 to 14 steps: the first step, the six-fold loop and each of its tails, in every number of blocks."""
    depth = {"forward": 64 * steps - 40, "dx": 64 * steps - 40, "i8": 128 * steps - 48}[op]
    if steps % 3 == 0:  # whole steps
        depth = (128 if op == "i8" else 64) * steps
    N, K = (depth, 8072) if op == "dx" else (8072, depth)
    _check_rows(op, "matmul_tile256", ALL_BLOCKS, N, K, op != "dx" and steps % 2 == 1,
                "f32" if steps % 4 < 2 else "bf16", steps)


@pytest.mark.parametrize("out_name", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["forward", "dx", "i8"])
@pytest.mark.parametrize("rows,kernel", [("many", "matmul_tile256_nt"), ("few", "matmul_tile128_nt")])
def test_streamed_weights(op, out_name, rows, kernel):
    """More than 256 MB of weights in whole lines: groups of one tile of rows, read once, beside one of several."""
    sizes = [60, 0, 250, 700, 33, 1] + [20] * 18 if rows == "many" else [8, 0, 1, 60, 131] + [0] * 19
    K = 5632 if op == "i8" else 2816
    _check_rows(op, kernel, sizes, 2024, K, op != "dx" and out_name == "f32", out_name, 50)


@pytest.mark.parametrize("K,start,kernel", [(2816, 0, "matmul_tile128_nt"), (2808, 0, "matmul_tile128"),
                                            (2816, 8, "matmul_tile128"), (2816, 64, "matmul_tile128_nt")])
def test_weights_are_streamed_in_whole_lines(K, start, kernel):
    """Rows that are not whole 128-byte lines, or that start inside one, share lines: those keep the default policy
    (streamed, they took up to a quarter longer)."""
    torch = _torch()
    sizes, N = [8, 0, 1, 60] + [0] * 20, 2024
    gen = torch.Generator(device="cuda")
    gen.manual_seed(53)
    off, d_off = _offsets(sizes)
    x, w = _ints(gen, int(off[-1]), K).bfloat16(), _ints(gen, len(sizes), N, K)
    big = torch.zeros(w.numel() + start, dtype=torch.bfloat16, device="cuda")
    big[start:] = w.view(-1)
    y, names = _launched(lambda: moe.moe_grouped_matmul(x, big[start:].view(w.shape), d_off))
    assert [k for k, _ in names] == [kernel]
    for g in range(len(sizes)):
        r = slice(int(off[g]), int(off[g + 1]))
        assert torch.equal(y[r], _exact(x[r], w[g].T, torch.bfloat16))


def _check_weights(sizes, N, K, gather, out_name, names, seed):
    torch = _torch()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    off, d_off = _offsets(sizes)
    rows, G = int(off[-1]), len(sizes)
    x_rows = rows // 3 if gather else rows
    dy, x = _ints(gen, rows, N), _ints(gen, x_rows, K)
    idx = torch.randint(0, x_rows, (rows,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    out_dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[out_name]
    out = torch.full((G, N, K), float("nan"), dtype=out_dtype, device="cuda")
    dyb, xb = dy.bfloat16(), x.bfloat16()

    def call():
        return moe.moe_grouped_matmul_dw(dyb, xb, d_off, row_index=idx, out=out)

    _, got = _launched(call)
    assert [k for k, _ in got] == names
    first = out.clone()
    xr = x if idx is None else x[idx.long()]
    for g in range(G):
        r = slice(int(off[g]), int(off[g + 1]))
        want = _exact(dy[r].T, xr[r], out_dtype)
        assert torch.equal(first[g], want), f"group {g}: {int((first[g] != want).sum())} values differ"
    for _ in range(3):
        call()
    assert torch.equal(out, first)


@pytest.mark.parametrize("out_name", ["bf16", "f32"])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
def test_weights_in_256_tiles(gather, out_name):
    """Groups of 0 to 14 steps of 64 rows, and rows that end inside a step, in one call."""
    sizes = [0, 1, 63, 64, 65, 130, 192, 250, 320, 384, 447, 512, 570, 640, 700, 769, 830, 896]
    _check_weights(sizes, 1000, 2024, gather, out_name, ["matmul_tile256"], 60)


@pytest.mark.parametrize("out_name", ["bf16", "f32"])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
def test_weights_in_256_tiles_of_cut_groups(gather, out_name):
    """One group holds most of the rows and is cut into ranges; the others are written at once."""
    sizes = [9000, 0, 1700, 1] + [331] * 15 + [334]
    _check_weights(sizes, 696, 696, gather, out_name, ["matmul_tile256", "matmul_join"], 61)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("long,gather", [("rows_in", False), ("rows_out", False), ("rows_out", True)],
                         ids=["rows_in", "rows_out", "rows_out_gathered"])
def test_rows_past_4_gib(long, dt, gather):
    """dy or x of more than 4 GiB, a long group that crosses the boundary and short ones wholly past it: all three
    products, exact (sums of at most 400,000 products of up to 2^4 stay below 2^24).  A gathered x is below 4 GiB."""
    torch = _torch()
    wide = 4096 if dt == "bf16" else 2048  # 8 KiB a row: row 524,288 is the first past 4 GiB
    N, K = (16, wide) if long == "rows_in" else (wide, 16)
    sizes = [300_000, 100, 299_900, 0, 101, 65, 3, 99_831]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    off, d_off = _offsets(sizes)
    rows, G = int(off[-1]), len(sizes)
    x_rows = 5000 if gather else rows
    x, dy, w = _ints(gen, x_rows, K), _ints(gen, rows, N), _ints(gen, G, N, K)
    idx = torch.randint(0, x_rows, (rows,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    xb, dyb, wb = x.to(dtype), dy.to(dtype), w.to(dtype)
    y = moe.moe_grouped_matmul(xb, wb, d_off, row_index=idx)
    dx = moe.moe_grouped_matmul_dx(dyb, wb, d_off)
    dw = moe.moe_grouped_matmul_dw(dyb, xb, d_off, row_index=idx, dw_dtype=moe.MOE_F32)
    xr = x if idx is None else x[idx.long()]
    for g in range(G):
        b, e = int(off[g]), int(off[g + 1])
        parts = [slice(b, e)] if e - b < 1000 else [slice(b, b + 300), slice(e - 300, e)]
        if b < 524_288 < e:
            parts.append(slice(524_288 - 200, 524_288 + 200))
        for r in parts:
            assert torch.equal(y[r], _exact(xr[r], w[g].T, dtype)), f"y, group {g}, rows {r}"
            assert torch.equal(dx[r], _exact(dy[r], w[g], dtype)), f"dx, group {g}, rows {r}"
        want = torch.zeros((N, K), dtype=torch.float64, device="cuda")
        for i in range(b, e, 50_000):
            r = slice(i, min(i + 50_000, e))
            want += dy[r].double().T @ xr[r].double()
        assert torch.equal(dw[g].double(), want), f"dw of group {g}"


@pytest.mark.parametrize("size", [(3, 120, 72, 56), (5, 600, 264, 136)])
def test_gradients_against_differences_along_their_signs(size):
    """As the product is linear, <dy, y(x + d) - y(x - d)> / 2 = <dx, d> without truncation error.  Along d = the
    sign of the formula's gradient the right side is the sum of its magnitudes, so that no wrong gradient comes
    near it: the bound is 2^-13 of that sum, and the fp32 roundings of both sides, of relative size
    sqrt(depth) 2^-24 and independent from output to output, are two orders below it."""
    torch = _torch()
    G, rows, N, K = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(12)
    cuts = np.sort(np.random.default_rng(4).integers(0, rows + 1, G - 1))
    off, d_off = _offsets(np.diff(np.concatenate([[0], cuts, [rows]])))
    x = torch.randn((rows // 3, K), generator=gen, device="cuda")
    w = torch.randn((G, N, K), generator=gen, device="cuda")
    dy = torch.randn((rows, N), generator=gen, device="cuda")
    idx = torch.randint(0, rows // 3, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    xr = x[idx.long()].contiguous()
    d, e = torch.zeros_like(xr), torch.zeros_like(w)
    for g in range(G):
        r = slice(int(off[g]), int(off[g + 1]))
        d[r] = torch.sign(dy[r].double() @ w[g].double()).float()
        e[g] = torch.sign(dy[r].double().T @ xr[r].double()).float()
    dx = moe.moe_grouped_matmul_dx(dy, w, d_off).double()
    plus, minus = (moe.moe_grouped_matmul(xr + s * d, w, d_off).double() for s in (1, -1))
    lhs, rhs = float(((plus - minus) / 2 * dy.double()).sum()), float((dx * d.double()).sum())
    assert rhs > 0 and abs(lhs - rhs) <= 2.0 ** -13 * lhs
    dw = moe.moe_grouped_matmul_dw(dy, x, d_off, row_index=idx).double()
    plus, minus = (moe.moe_grouped_matmul(x, w + s * e, d_off, row_index=idx).double() for s in (1, -1))
    lhs, rhs = float(((plus - minus) / 2 * dy.double()).sum()), float((dw * e.double()).sum())
    assert rhs > 0 and abs(lhs - rhs) <= 2.0 ** -13 * lhs


# --------------------------------------------------------------------------- very many output tiles
@pytest.mark.parametrize("op,depth,kernel", [
    ("forward", 8, "matmul_tile128"), ("dx", 8, "matmul_tile128_nt"), ("i8", 16, "matmul_tile128"),
    ("forward", 1, "matmul_any128"), ("dx", 1, "matmul_any128"), ("i8", 1, "matmul_any128")])
def test_rows_of_four_million_tiles(op, depth, kernel):
    """513 groups of 8192 tiles each: more work-groups than one row of the grid holds."""
    sizes = [1, 2, 0] + [1] * 510
    N, K = (depth, 1 << 20) if op == "dx" else (1 << 20, depth)
    # dx, depth 1: rows of W are whole 16-byte pieces, rows of dy (one value) are not
    _check_rows(op, kernel, sizes, N, K, op != "dx", "bf16", 70)


@pytest.mark.parametrize("K,kernel", [(8, "matmul_tile128"), (1, "matmul_any64")])
def test_weights_of_four_million_tiles(K, kernel):
    _check_weights([1, 2, 0] + [1] * 510, 1 << 20, K, True, "bf16", [kernel], 71)


@pytest.mark.parametrize("rows,cols", [((1 << 24) + 5, 8), ((1 << 22) + 3, 2056)])
def test_quantize_more_rows_than_a_grid_row(rows, cols):
    torch = _torch()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    x = _ints(gen, rows, cols, top=127).bfloat16()
    x[:, cols - 1] = -127  # the codes are then the values themselves
    codes, scales = moe.moe_quantize_rows(x)
    assert bool((scales == 1).all())
    for i in range(0, rows, 1 << 20):
        assert torch.equal(codes[i:i + (1 << 20)].bfloat16(), x[i:i + (1 << 20)])


def test_output_types_that_contradict_each_other_are_refused():
    torch = _torch()
    x = torch.ones((4, 16), device="cuda").bfloat16()
    w = torch.ones((1, 8, 16), device="cuda").bfloat16()
    q, s = moe.moe_quantize_rows(x)
    qw, sw = torch.ones((1, 8, 16), dtype=torch.int8, device="cuda"), torch.ones((1, 8), device="cuda")
    for dtype, other in ((torch.float32, moe.MOE_BF16), (torch.bfloat16, moe.MOE_F32)):
        y, dx = torch.zeros((4, 8), device="cuda", dtype=dtype), torch.zeros((4, 16), device="cuda", dtype=dtype)
        dw = torch.zeros((1, 8, 16), device="cuda", dtype=dtype)
        for bad in (lambda: moe.moe_matmul_i8(q, s, qw, sw, y_dtype=other, out=y),
                    lambda: moe.moe_grouped_matmul(x, w, None, y_dtype=other, out=y),
                    lambda: moe.moe_grouped_matmul_dx(w[0, :4, :8].contiguous(), w, None, dx_dtype=other, out=dx),
                    lambda: moe.moe_grouped_matmul_dw(w[0, :4, :8].contiguous(), x, None, dw_dtype=other, out=dw)):
            with pytest.raises(ValueError):
                bad()
        assert not bool(y.any()) and not bool(dx.any()) and not bool(dw.any())
        assert moe.moe_matmul_i8(q, s, qw, sw, out=y) is y and bool((y == 16).all())
    assert moe.moe_matmul_i8(q, s, qw, sw).dtype == torch.bfloat16
    assert moe.moe_matmul_i8(q, s, qw, sw, y_dtype=moe.MOE_F32).dtype == torch.float32
