"""What of the matrix products can be run without a GPU, compiled by nvcc into a program
for the host: how a tile's k is cut into segments, how they are added up, and what a wait
that gives up leaves."""

import subprocess

import pytest

from gradient_synchronisation_gb300 import _build

SOURCE = r"""
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include "product.cuh"

namespace zr {
int sm_count() { return 152; }
}  // namespace zr

// parts, half, the first segment whose wait gives up (-1: none): v[0], v[half - 1], whether
// the half row's sum is NaN, what sum_segments returned and how many segments were taken.
static void sum(int parts, int half, int fails) {
  float v[128];
  int g = 0, taken = 0;
  const bool ok = zr::sum_segments(
      v, parts, half, true, [&]() { return g != fails; },
      [&](int c, float* u) {
        for (int k = 0; k < 32; ++k) u[k] = (float)((g + 1) * (c + k + 1));
      },
      [&]() { ++taken, ++g; });
  float all = 0.f;
  for (int k = 0; k < half; ++k) all += v[k];
  printf("%g %g %d %d %d\n", v[0], v[half - 1], (int)std::isnan(all), (int)ok, taken);
}

int main(int n, char** args) {
  if (n == 4) sum(atoi(args[1]), atoi(args[2]), atoi(args[3]));
  else
    for (int k = 0; k <= atoi(args[1]); ++k) printf("%d\n", zr::segment_steps(k, atoi(args[2])));
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("product")
    (at / "host.cu").write_text(SOURCE)
    out = str(at / "host")
    res = subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-I", _build.INCLUDE, "-I", _build.CSRC, "-o", out,
                          str(at / "host.cu")], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr

    def run(*args):
        return subprocess.run([out, *map(str, args)], capture_output=True, text=True, check=True).stdout.split()

    return run


@pytest.mark.parametrize("parts, half", [(1, 64), (2, 64), (5, 128)])
def test_a_wait_that_gives_up_leaves_no_sum(program, parts, half):
    """Whichever segment's it is: the sum of those before it would be finite and wrong."""
    terms = parts * (parts + 1) // 2
    assert program(parts, half, -1) == [str(terms), str(terms * half), "0", "1", str(parts)]
    for fails in range(parts):
        got = program(parts, half, fails)
        assert got[0] == "nan" and got[2:] == ["1", "0", str(fails)], fails


@pytest.mark.parametrize("rows, most", [(1, 2), (128, 2), (129, 8), (4096, 8)])
def test_segments_have_at_most_their_terms(program, rows, most):
    """Steps of 64 terms: 128 terms to a segment for few rows at every depth, 512 for
    many, and two segments at least where there are more than four steps."""
    steps = [int(v) for v in program(300, rows)]
    assert steps[0] == 1
    for k, n in enumerate(steps[1:], 1):
        assert 1 <= n <= most, k
        parts = -(-k // n)
        assert (parts - 1) * n < k and parts <= max(-(-k // most) + 1, 2), k
        assert k <= 4 or parts >= 2, k
