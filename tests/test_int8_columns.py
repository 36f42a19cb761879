"""The columns that the threads of an 8-bit row take, walked on the host: each
vector of eight once, none outside the row, up to the longest row accepted."""
import subprocess

import pytest

from w4a16_grouped_moe_amd.build import CSRC

PROGRAM = r"""
#include "int8_columns.hpp"
#include <cstdio>
#include <cstdlib>

// 512 threads, eight values each, the first four vectors kept elsewhere: the
// form that the longest rows take
int main(int, char **argv)
{
    const int end = (int)strtoll(argv[1], nullptr, 10);
    long long vectors = 0, sum = 0;
    for (int tid = 0; tid < 512; ++tid) {
        long long want = (4 * 512 + tid) * 8LL;
        dgw4::each_column<512 * 8>((int)want, end, [&](int k) {
            if (k != want || k >= end) {
                printf("thread %d: column %d where %lld was due\n", tid, k, want);
                fflush(stdout);
                _Exit(1);
            }
            want += 512 * 8;
            ++vectors;
            sum += k;
        });
    }
    printf("%lld %lld\n", vectors, sum);
    return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("columns")
    src, exe = d / "walk.cpp", d / "walk"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", f"-I{CSRC}", "-o", str(exe), str(src)], check=True)
    return lambda end: subprocess.run([str(exe), str(end)], capture_output=True, text=True, timeout=60)


@pytest.mark.parametrize("end", [1, 16384, 16385, 70016, 2**31 - 8192, 2**31 - 4097, 2**31 - 4096, 2**31 - 4089,
                                 2**31 - 2049, 2**31 - 17, 2**31 - 16])
def test_each_vector_once(walk, end):
    r = walk(end)
    assert r.returncode == 0, r.stdout
    first = 4 * 512 * 8
    n = max(0, -(-(end - first) // 8))                     # vectors of columns first, first + 8, ...
    assert [int(v) for v in r.stdout.split()] == [n, n * first + 8 * (n * (n - 1) // 2)]
