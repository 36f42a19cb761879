"""Which tile an 8-bit product runs on, asked on the host: the sizes that the GPU
tests give each tile do reach it, and every choice is one that can be launched."""
import subprocess

import pytest

from tests import test_gpu_int8
from w4a16_grouped_moe_amd.build import CSRC

PROGRAM = r"""
#include "int8_tiles.hpp"
#include <cstdio>

int main()
{
    int T, K, N;
    while (scanf("%d %d %d", &T, &K, &N) == 3) {
        const int i = dgw4::pick_tile(T, K, N);
        const dgw4::I8Tile &t = dgw4::kTiles[i];
        const long long groups = ((N + (long long)t.bn - 1) / t.bn) * ((T + (long long)t.bt - 1) / t.bt);
        printf("%d %d %lld\n", i, (int)(sizeof(dgw4::kTiles) / sizeof(t)), groups * t.threads);
    }
}
"""


@pytest.fixture(scope="module")
def pick(tmp_path_factory):
    d = tmp_path_factory.mktemp("tiles")
    src, exe = d / "tiles.cpp", d / "tiles"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", f"-I{CSRC}", "-o", str(exe), str(src)], check=True)

    def ask(shapes):
        text = "\n".join(" ".join(map(str, s)) for s in shapes)
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60, check=True)
        return [tuple(int(v) for v in line.split()) for line in r.stdout.split("\n") if line]
    return ask


def _shapes(test):
    mark, = [m for m in test.pytestmark if m.name == "parametrize" and m.args[0] == "T,K,N"]
    return mark.args[1]


def test_every_tile_has_its_gpu_tests(pick):
    shapes = _shapes(test_gpu_int8.test_product_tiles) + _shapes(test_gpu_int8.test_product_tiles_in_parts)
    got = pick(shapes)
    # two sizes at least for each tile, with K in whole stages of all its parts
    # and not
    parts = {3: 2, 4: 2, 5: 2, 6: 2, 7: 2, 8: 4}
    for tile in range(got[0][1]):
        ks = [s[1] for s, g in zip(shapes, got) if g[0] == tile]
        assert len(ks) >= 2, tile
        assert any(k % (128 * parts.get(tile, 1)) for k in ks), tile
    assert {4, 8} <= {g[0] for s, g in zip(shapes, got) if s[1] % (128 * parts.get(g[0], 1)) == 0}
    # and both forms of the largest: one tile of tokens, and more
    assert {s[0] <= 256 for s, g in zip(shapes, got) if g[0] == 0} == {True, False}


@pytest.mark.parametrize("T,K,N", [(1, 16, 2**31 - 257), (2**31 - 257, 16, 1), (1, 131056, 2**31 - 257),
                                   (1, 16, 2**29 + 17), (256, 16, 2**29), (2**31 - 257, 16, 32)])
def test_launches_stay_under_2_to_the_32(pick, T, K, N):
    (tile, tiles, threads), = pick([(T, K, N)])
    assert 0 <= tile < tiles and threads < 2**32
