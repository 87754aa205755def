"""A sequence's tokens from what the caller's arrays say, whatever that is: the function that the
kernels call, compiled for the host."""
import os
import subprocess

import pytest

from bit_quantized_gemv_amd import build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ops_cache.hpp"

int main()
{
    const int ends[] = {-2147483647 - 1, -2147483647, -8, -1, 0, 1, 3, 6, 7, 8, 100, 4194304, 2147483640, 2147483647};
    int bad = 0;
    for (int T : {1, 7, 4194304})
        for (int places : {0, 1, 30, 1 << 30})
            for (int s0 : ends)
                for (int s1 : ends)
                    for (int n : ends) {
                        const int starts[] = {s0, s1}, lengths[] = {n};
                        ops::Cache c = {};
                        c.starts = starts;
                        c.lengths = lengths;
                        c.max_places = places;
                        c.T = T;
                        const ops::Seq s = ops::sequence(c, 0);
                        const auto within = [](long long x, long long top) { return x < 0 ? 0 : x > top ? top : x; };
                        const long long from = within(s0, T), to = within(s1, T);
                        if (s.start != from || s.count != within(to - from, T) || s.length != within(n, places)) {
                            if (bad++ < 5) printf("T %d starts %d %d: from %d, %d tokens\n", T, s0, s1, s.start, s.count);
                        }
                    }
    printf("%d\n", bad);
    return bad != 0;
}
"""


def test_sequences_stay_in_the_arrays(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    src, exe = tmp_path / "sequence.hip", tmp_path / "sequence"
    src.write_text(PROGRAM)
    subprocess.run([build.HIPCC, "--offload-host-only", "-O2", "-std=c++17", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"), "-o", str(exe),
                    str(src)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
