"""How the rows of a batch's logits are cut into workgroups, asked on the host:
every row and column has one, a launch stays within its limits, and the GPU tests'
sizes have workgroups of several rows in every form."""
import random
import subprocess

import pytest

from tests import entropy_bound
from tests import test_gpu_logit_rows as rows
from w4a16_grouped_moe_amd.build import CSRC

PROGRAM = r"""
#include "logit_cut.hpp"
#include <cstdio>

int main()
{
    int R, V, max_tokens, shared;
    while (scanf("%d %d %d %d", &R, &V, &max_tokens, &shared) == 4) {
        const int threads = max_tokens >= dgw4::kLongHistory ? dgw4::kBroad : dgw4::kNarrow;
        const int e = dgw4::per_thread(R, V);
        const dgw4::Cut c = dgw4::cut(R, V, dgw4::tile_of(threads, e), shared != 0);
        printf("%d %d %d %d %u\n", threads, e, c.tiles, c.rows, c.groups);
    }
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    d = tmp_path_factory.mktemp("cut")
    src, exe = d / "cut.cpp", d / "cut"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", f"-I{CSRC}", "-o", str(exe), str(src)], check=True)

    def ask(shapes):
        text = "\n".join(" ".join(map(str, s)) for s in shapes)
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60, check=True)
        return [tuple(int(v) for v in line.split()) for line in r.stdout.split("\n") if line]
    return ask


def test_gpu_tests_have_workgroups_of_several_rows(cut):
    got = cut([(*s, 1) for s in rows.ROWS])
    assert all(g[3] > 1 for g in got)
    assert {g[:2] for g in got} == {(256, 8), (256, 16), (512, 8), (512, 16)}
    # tiles that end before the row does, but where the sizes that take 8 columns a
    # thread and 512 threads have one tile only; and more than two rows
    for form in ((256, 8), (256, 16), (512, 16)):
        assert any(g[:2] == form and V > g[0] * g[1] for g, (_, V, _) in zip(got, rows.ROWS))
    for form in ((256, 16), (512, 16)):
        assert any(g[:2] == form and g[3] > 2 for g in got)
    # own sequences: several rows only where the grid would be too long
    (_, _, _, several, _), = cut([(5_000_003, 40, 3, 0)])
    assert several > 1


def test_cuts(cut):
    rng = random.Random(4)
    shapes = [(2**31 - 1, 1, 0, 0), (2**31 - 1, 511, 0, 1), (1, 2**30 - 1, 0, 0), (1024, 2**30 - 1, 20000, 1)]
    while len(shapes) < 30000:
        R, V = int(2 ** rng.uniform(0, 31)) - 1, int(2 ** rng.uniform(0, 30))
        if 1 <= R and 1 <= V and R * V < 2**40:
            shapes.append((R, V, rng.choice([0, 16383, 16384]), rng.randint(0, 1)))
    for (R, V, max_tokens, shared), (threads, e, tiles, several, groups) in zip(shapes, cut(shapes)):
        tile = threads * e
        assert tiles * tile >= V > (tiles - 1) * tile
        assert several >= 1 and groups == -(-R // several) * tiles and groups * threads < 2**32
        # the workspace has the parts of the wider workgroup's cut
        assert tiles * (threads // 64) <= -(-V // (512 * e)) * 8
        assert (e, tiles * (threads // 64)) == entropy_bound.cut(R, V, max_tokens)
