"""How many CTAs a large fork's cluster has where the GPU, or the part of it that a process has, cannot place sixteen."""
import os
import subprocess

from block_sparse_long_pool_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_sparse_long_pool_gb300", "csrc")

HARNESS = r"""
#include <cstdio>
#include "paged.cuh"

int main()
{
    for (int room = 0; room <= 20; ++room)
        printf("%d ", sp_host::largest_cluster(16, [&](int n) { return n <= room; }));
    int asked = 0;
    sp_host::largest_cluster(16, [&](int) { ++asked; return false; });
    printf("%d", asked);
    return 0;
}
"""


def test_the_largest_cluster_that_fits(tmp_path):
    src, exe = tmp_path / "harness.cu", tmp_path / "harness"
    src.write_text(HARNESS)
    cmd = [build.nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    out = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert out == [1, 1, 2, 2] + [4] * 4 + [8] * 8 + [16] * 5 + [4]   # a single CTA is not asked for: it always fits
