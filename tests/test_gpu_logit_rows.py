"""GPU: the rules on logits where a workgroup takes several rows in turn and keeps
what it made of their sequence (tests/test_logit_cut.py asks the library's own
arithmetic that it does for the sizes here), for every width of workgroup and
number of columns a thread takes."""
import numpy as np
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import entropy_bound, rules_ref
from tests.few_ref import same_bits

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    dg.lib()


def _dev(u):
    return dg.LogitRules(**{k: v.cuda() for k, v in u.items()})


# R, V, max_tokens
ROWS = [
    (1100, 3000, 3000), (1360, 2100, 2100),              # 256 threads, 8 columns each
    (1000, 9000, 9000), (2100, 9001, 9001), (4200, 4500, 4500),       # 256, 16
    (3000, 1000, 16384),                                 # 512, 8
    (1500, 20011, 20011), (2100, 8193, 16400),           # 512, 16
]


def _shared(rng, R, V, L, order, mask):
    """Rules of sequences from no token to all of them, scattered and side by side,
    each with many rows: next to each other, in any order, some with none."""
    runs = [min(n, V) for n in (0, 1, 63, 64, 65, 127, 128, 129, 130, 500, 1024, V)]
    S = 2 * len(runs)
    u = rules_ref.random_rules(rng, S, V, L=L, bias=7)
    for i, n in enumerate(runs):
        near = min(1024, V)
        u["tokens"][2 * i, :n] = torch.from_numpy(rng.permutation(near)[:n] if n <= near else rng.permutation(V)).int()
        u["tokens"][2 * i + 1, :n] = torch.arange(n).int()
        u["lengths"][2 * i:2 * i + 2] = n
    u["prompt_lengths"] = u["lengths"] // 2
    seq = rng.integers(-1, S + 1, R)
    u["row_seq"] = torch.from_numpy(np.sort(seq) if order == "sorted" else seq).int()
    if mask:
        M = 24
        bits = rng.integers(0, 2 ** 32, (M, (V + 31) // 32), dtype=np.uint64).astype(np.uint32).view(np.int32)
        bits[0], bits[1] = 0, -1
        u["mask"] = torch.from_numpy(bits)
        u["mask_row"] = torch.from_numpy(rng.integers(-1, M + 1, R).astype(np.int32))
    return u


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("order,mask", [("sorted", True), ("any", False)])
@pytest.mark.parametrize("R,V,L", ROWS)
def test_several_rows_of_a_sequence(R, V, L, order, mask, dtype):
    rng = np.random.default_rng([R, V, mask])
    u = _shared(rng, R, V, L, order, mask)
    l = torch.from_numpy((rng.standard_normal((R, V)) * 3).astype(np.float32))
    l[torch.from_numpy(rng.random((R, V)) < 0.01)] = float("-inf")
    l = l.to(dtype)
    rules, want = _dev(u), rules_ref.adjusted(l, u)
    # rows apart, from an odd element on
    wide = torch.zeros((R, V + 6), dtype=dtype, device="cuda")
    x = wide[:, 3:V + 3]
    x.copy_(l)
    assert same_bits(dg.adjust_logits(x, rules), torch.from_numpy(want))
    assert same_bits(dg.adjust_logits(x, rules, dtype=dtype), torch.from_numpy(want).to(dtype))
    h, smp, am = dg.sample_adjusted(x, rules, R + V)
    rules_ref.check_sample(want, R + V, None, smp, am)
    entropy_bound.check(h, want, L)
    h2, none, am2 = dg.sample_adjusted(x, rules, draw=False)
    assert same_bits(h, h2) and torch.equal(am, am2)
    assert same_bits(x, l)
    # in place: all of the row with a scale, without one only what changes
    y = x.clone()
    dg.adjust_logits(y, rules, out=y)
    assert same_bits(y, torch.from_numpy(want).to(dtype))
    plain = {k: v for k, v in u.items() if k != "scale"}
    dg.adjust_logits(x, _dev(plain), out=x)
    assert same_bits(x, torch.from_numpy(rules_ref.adjusted(l, plain)).to(dtype))
    assert not wide[:, :3].any() and not wide[:, V + 3:].any()


def test_several_rows_of_own_sequences():
    # more rows than a grid has workgroups: one workgroup's rows each bring a sequence
    R, V, L = 5_000_003, 40, 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-8, 9, (R, V), device="cuda", generator=gen).to(F16)
    tokens = torch.randint(0, V, (R, L), device="cuda", dtype=torch.int32, generator=gen)
    lengths = torch.randint(0, L + 1, (R,), device="cuda", dtype=torch.int32, generator=gen)
    presence = torch.randint(1, 9, (R,), device="cuda", generator=gen).float()
    rules = dg.LogitRules(tokens=tokens, lengths=lengths, presence=presence)
    seen = torch.zeros((R, V + 1), dtype=torch.bool, device="cuda")
    live = torch.arange(L, device="cuda") < lengths[:, None]
    seen.scatter_(1, torch.where(live, tokens, torch.full_like(tokens, V)).long(), True)
    want = torch.where(seen[:, :V], x.float() - presence[:, None], x.float())     # whole numbers: exact
    got = dg.adjust_logits(x, rules)
    assert torch.equal(got, want)
    top = want.amax(1, keepdim=True)
    first = torch.where(want == top, torch.arange(V, device="cuda"), V).amin(1)
    assert torch.equal(dg.sample_adjusted(x, rules, draw=False, entropy=False)[2].long(), first)
    dg.adjust_logits(x, rules, out=x)
    assert torch.equal(x, want.to(F16))
