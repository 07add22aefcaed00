"""The row that a route reads, on the host: the header that the grouped products' kernels share, compiled
as plain C++ (CPU only)."""
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "quantized_expert_grouped_amd", "csrc")
MAIN = r"""
#include <stdio.h>
#include "route_row.hpp"
int main() {
  int K, route, n_act;
  while (scanf("%d %d %d", &K, &route, &n_act) == 3) {
    const moe::Division d = moe::division_by(K);
    printf("%d\n", moe::route_row(route, d.mul, d.shift, n_act));
  }
}
"""


@pytest.fixture(scope="module")
def rows(tmp_path_factory):
    at = tmp_path_factory.mktemp("route_row")
    (at / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(at / "main.cpp"), "-o", str(at / "main")],
                   check=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(at / "main")], input=text, capture_output=True, text=True, check=True)
        return [int(v) for v in out.stdout.split()]

    return ask


def around(K):
    """The range's ends, both sides of its powers of two and of the multiples of K near them."""
    top = 2 ** 31 - 1
    near = {0, 1, K - 1, K, top, top - 1, top // K * K, top // K * K - 1}
    for p in range(20, 32):
        m = 2 ** p // K * K
        near |= {2 ** p - 1, 2 ** p, m - 1, m, m + K - 1, m + K, m + 2 * K - 1}
    rng = np.random.default_rng(K)
    near |= {int(v) // K * K + j for v in rng.integers(0, 2 ** 31, 200) for j in (-1, 0)}
    return sorted(r for r in near if 0 <= r <= top)


def test_every_route_reads_its_own_row(rows):
    """The quotient is exact over all of int32: activations of as many rows as routes can name."""
    cases = [(K, r, 2 ** 31 - 1) for K in range(1, 65) for r in around(K)]
    assert rows(cases) == [min(r // K, n - 1) for K, r, n in cases]


def test_strays_read_the_nearest_row(rows):
    cases = [(K, r, n) for K in range(1, 65) for n in (1, 3, 8192, 1 << 26)
             for r in around(K) + [-1, -5, -2 ** 31, -2 ** 31 + 1]]
    got = rows(cases)
    assert got == [min(max(r, 0) // K, n - 1) for K, r, n in cases]
    assert all(0 <= row < n for row, (_, _, n) in zip(got, cases))
