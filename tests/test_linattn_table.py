"""The places of packed sequences in the chunk table: inside it for any offsets,
also out of order, where the chunks that they name add up to more than 2^31."""
import shutil
import subprocess

import pytest

from gated_delta_rule_47_gb300 import build

MAIN = r"""
#include "linattn.cuh"
#include <cstdio>
int main() {
    for (long long at : {0LL, 5LL, 99LL, 100LL, 101LL, 2147483647LL, 2147483648LL, 2560000000LL, 4294967296LL, 65534LL << 24})
        for (int n : {0, 1, 64, 1 << 24}) {
            const int2 p = gdn::la::in_table(at, n, 100);
            printf("%lld %d %d %d\n", at, n, p.x, p.y);
        }
}
"""


@pytest.mark.skipif(not shutil.which("nvcc") and not shutil.which("/usr/local/cuda/bin/nvcc"), reason="needs nvcc")
def test_places(tmp_path):
    src, exe = tmp_path / "places.cu", tmp_path / "places"
    src.write_text(MAIN)
    subprocess.run([build.nvcc(), *build.FLAGS, str(src), "-o", str(exe)], check=True)
    rows = [tuple(map(int, line.split())) for line in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()]
    assert len(rows) == 40
    for at, n, first, count in rows:
        assert (first, count) == (min(at, 100), max(min(n, 100 - at), 0))
