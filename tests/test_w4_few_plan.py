"""How a few-token W4A16 call is cut up, asked on the host: every plan covers its
channels and K and can be launched, and the GPU tests' sizes reach every form."""
import random
import subprocess

import pytest

from tests import test_gpu_w4_few_forms as forms
from w4a16_grouped_moe_amd.build import CSRC

PROGRAM = r"""
#include "w4_few_plan.hpp"
#include <cstdio>

int main()
{
    int T, K, N, g;
    while (scanf("%d %d %d %d", &T, &K, &N, &g) == 4) {
        int tokens;
        const int i = dgw4::form_of(T, K, N, g, tokens);
        const dgw4::Form &f = dgw4::kForms[i];
        const dgw4::Plan p = dgw4::plan_of(f, tokens, K, N);
        printf("%d %d %d %d %d %u %d %d %d %d %d %d %d %zu\n", i, p.split, p.turns, p.batches, p.tokens, p.magic,
               f.waves, f.tb, f.cb, f.m, f.resident, f.max_split, f.step, dgw4::lds_of(f, tokens, K, g));
    }
}
"""
NAMES = ("form split turns batches tokens magic waves tb cb m resident max_split step lds").split()


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", f"-I{CSRC}", "-o", str(exe), str(src)], check=True)

    def ask(shapes):
        text = "\n".join(" ".join(map(str, s)) for s in shapes)
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60, check=True)
        return [dict(zip(NAMES, map(int, line.split()))) for line in r.stdout.split("\n") if line]
    return ask


def _key(p):
    return p["form"], p["split"], p["turns"] > p["resident"]


def _chunks(K, p):
    return -(-K // (512 * p["m"]))


@pytest.mark.parametrize("name,groups", [("SHAPES", (64, 128)), ("RAGGED", (64,))])
def test_every_form_has_its_gpu_tests(plan, name, groups):
    shapes = getattr(forms, name)
    for g in groups:
        got = plan([(*s, g) for s in shapes])
        every = {(p["form"], s, several) for p in got for s in range(0, p["max_split"] + 1, p["step"])
                 for several in (False, True)}
        assert len(every) == 36
        assert every == {_key(p) for p in got}
        # x in three chunks or more in every form that has chunks; where two lie
        # ready, in an odd and in an even number of them
        chunks = {}
        for (T, K, N), p in zip(shapes, got):
            if p["m"]:
                chunks.setdefault(_key(p), set()).add(_chunks(K, p))
        assert len(chunks) == 18 and all(max(c) >= 3 for c in chunks.values())
        if name == "SHAPES":
            for k in ((2, 4), (3, 1), (3, 2), (4, 1), (4, 2)):
                c = chunks[(*k, False)] | chunks[(*k, True)]
                assert {v % 2 for v in c} == {0, 1}, k


def test_plans_cover_their_calls(plan):
    rng = random.Random(3)
    shapes = [(1, 64, 1, 64), (64, 1 << 24, 1, 64), (64, 1 << 24, 2**31 - 257, 128), (1, 64, 2**31 - 257, 64)]
    for _ in range(30000):
        g = rng.choice([64, 128])
        shapes.append((rng.randint(1, 64), g * int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(0, 30)), g))
    for (T, K, N, g), p in zip(shapes, plan(shapes)):
        parts = 1 << p["split"]
        assert 1 <= p["tokens"] <= min(T, 16 * p["tb"]) and parts <= p["waves"]
        channels = (p["waves"] >> p["split"]) * 16 * p["cb"]          # of a turn
        assert p["turns"] * channels >= N > (p["turns"] - 1) * channels
        # a wave's batches of 512 columns
        assert p["batches"] * 512 * parts >= K
        if p["m"] == 0:
            static = p["waves"] * p["cb"] * 1024
            assert p["lds"] + static <= 160 * 1024
            for i in {0, K // 8 - 1, K // 8, p["tokens"] * (K // 8) - 1}:
                assert i * p["magic"] >> 32 == i // (K // 8)
        else:
            assert p["waves"] * p["tb"] * p["cb"] * 1024 <= p["lds"] <= 160 * 1024
            # a turn stores each chunk once, its last one before its last group, and
            # where two lie ready whole pairs of them in each batch
            depth = 2 if 2 * p["m"] <= parts else 1
            chunks = -(-_chunks(K, p) // depth) * depth
            assert (chunks - 1) * p["m"] < p["batches"] * parts
            assert parts // p["m"] % depth == 0
        assert -(-T // p["tokens"]) <= 4
