"""The move counts of mla_cache_evict stay in 32 bits (no GPU needed): the rule
for how many requests are counted at once, compiled as host code."""
import subprocess

from mla_latent_kv_cache_gb300 import build as mbuild

PROGRAM = r"""
#include "launch.cuh"
#include <cstdio>
int main() {
    const int lens[] = {0, 1, 2, 4160, 262144, 5592403, 5592404, 5592405, 5592406, 5592407, 16777216, 1 << 29, (1 << 30) - 1, 1 << 30};
    for (int n : lens) std::printf("%d %d\n", n, mla::evict_requests_at_once(n));
}
"""


def test_the_sum_of_the_moves_counted_at_once_fits_32_bits(tmp_path):
    src, exe = tmp_path / "rule.cpp", tmp_path / "rule"
    src.write_text(PROGRAM)
    subprocess.run([mbuild.nvcc(), "-std=c++17", "-I", mbuild.CSRC, str(src), "-o", str(exe)], check=True)
    rows = [tuple(map(int, r.split())) for r in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    assert len(rows) == 14
    for n, reqs in rows:
        most = n // 2  # rows that a request of n tokens can move
        assert 1 <= reqs <= 1536
        assert reqs * most < 2 ** 32
        assert reqs == 1536 or (reqs + 1) * most >= 2 ** 32 - most  # and no fewer than need be
