"""The norm of more rows than one dimension of a launch takes."""
import pytest

import moe_layer_forward_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def test_rows_past_2_to_the_22_of_a_work_group_each():
    """Rows of 8200 values have 1024 lanes, so that 2^22 rows have 2^32 threads: 69 GB, normed in place.  A row's 1 / sqrt is
    off by at most (62 + 1) / 2 + 4 u, y two products later by less than 40 u and its rounding."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.empty_cache()
    rows, cols = (1 << 22) + 3, 8200
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    parts = [slice(a, a + 4) for a in (0, (1 << 21) - 2, (1 << 22) - 2)] + [slice(rows - 2, rows)]
    for p in parts:
        x[p] = torch.randn(x[p].shape, generator=gen, device="cuda").bfloat16()
    h = [x[p].double() for p in parts]
    w = torch.randn(cols, generator=gen, device="cuda")
    assert moe.moe_rms_norm(x, w, out=x) is x
    for p, v in zip(parts, h):
        ref = v / ((v * v).mean(dim=1, keepdim=True) + 1e-6).sqrt() * w.double()
        assert bool(((x[p].double() - ref).abs() <= (2.0 ** -8 + 40 * U) * ref.abs() + 2.0 ** -126).all())
    assert not bool(x[(1 << 22) - 12:(1 << 22) - 2].any()) and not bool(x[(1 << 21) + 2:(1 << 21) + 12].any())
    del x
    torch.cuda.empty_cache()
