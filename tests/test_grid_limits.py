"""The grids of large launches, on the host: a dimension has fewer than 2^32 threads."""
import subprocess

from moe_layer_forward_amd import build

PROGRAM = """
#include <cstdio>
#include "gmm.h"
int main() {
  long long n;
  while (scanf("%lld", &n) == 1) {
    const dim3 g = moe::gmm_grid(n);
    printf("%u %u %u\\n", g.x, g.y, g.z);
  }
}
"""


def _grids(tmp_path, counts):
    src, exe = tmp_path / "grid.cpp", tmp_path / "grid"
    src.write_text(PROGRAM)
    subprocess.run([build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", f"-I{build.CSRC}", str(src), "-o",
                    str(exe)], check=True, capture_output=True)
    out = subprocess.run([str(exe)], input=" ".join(map(str, counts)), check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_a_dimension_has_fewer_than_2_to_the_32_threads(tmp_path):
    """Work-groups of up to 1024 threads (a norm's, one long row each), of one, four and sixteen rows, around every border."""
    rows = [1, 7, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, (1 << 22) - 1, 1 << 22, (1 << 22) + 5, 1 << 25, (1 << 31) - 1]
    counts = sorted({-(-r // per) for r in rows for per in (1, 4, 16)} | {(1 << 32) - 1})
    grids = _grids(tmp_path, counts)
    assert len(grids) == len(counts)
    for n, (x, y, z) in zip(counts, grids):
        assert x * 1024 < 1 << 32, (n, x)
        assert z == 1 and y <= 65535 and x * y >= n and x * (y - 1) < n
        assert y == 1 or x % 8 == 0  # work-group n on XCD n % 8

