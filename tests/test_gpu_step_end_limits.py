"""GPU: the operators at the end of a step at the ends of what they accept: the
longest K, the most channels and columns, the highest count, rules and logits of any
value, scales and zero points at their type's ends; the rules in place in a captured
graph whose rows share sequences."""
import numpy as np
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import rules_ref
from tests.few_ref import same_bits
from tests.test_gpu_w4_few_forms import _reference, _weights

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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _close(y, x, w, g):
    want, bound = _reference(x, *w, g, y.dtype)
    err = (y.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("T,N,xt", [(1, 3, F16), (16, 16, BF16), (33, 40, F16)])
def test_longest_k(T, N, xt):
    gen = _gen(T)
    K = 1 << 24
    x = torch.randn((T, K), device="cuda", generator=gen).to(xt)
    for g in (64, 128):
        w = _weights(gen, N, K, g)
        y = dg.w4a16_linear_few(x, (*w, g), dtype=F32)
        _close(y, x, w, g)
        if N % 16 == 0:
            assert same_bits(dg.w4a16_linear_few(x, dg.pack_tiled((*w, g)), dtype=F32), y)


def test_most_channels():
    # 2^31 - 257 channels of K = 64: 69 GB of codes
    N, K, g = 2**31 - 257, 64, 64
    gen = _gen(3)
    q = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    q.view(-1).random_(0, 256, generator=gen)
    s = torch.empty((N, 1), dtype=F16, device="cuda").uniform_(0.005, 0.02, generator=gen)
    z = torch.empty((N, 1), dtype=F16, device="cuda").random_(0, 16, generator=gen)
    x = torch.randn((2, K), device="cuda", generator=gen).to(BF16)
    y = dg.w4a16_linear_few(x, (q, s, z, g))
    for n in (0, 2**26 - 20, 2**27 - 20, 2**30 - 20, N - 3000, N - 40):
        part = slice(n, n + 40)
        _close(y[:, part], x, [v[part] for v in (q, s, z)], g)


@pytest.mark.parametrize("xt", [F16, BF16], ids=str)
def test_scales_and_zero_points_at_their_ends(xt):
    gen = _gen(4)
    f = torch.finfo(F16)
    T, K, N, g = 9, 512, 96, 64
    x = torch.randn((T, K), device="cuda", generator=gen).to(xt)
    q, s, z = _weights(gen, N, K, g)
    s[:, 0], s[:, 1], s[:, 2], s[:, 3] = f.max, f.smallest_normal / 1024, f.smallest_normal / 2, 0
    z[::3, 4], z[1::3, 4], z[2::3, 4] = f.max, f.min, f.smallest_normal / 1024
    z[:, 5] = -16
    _close(dg.w4a16_linear_few(x, (q, s, z, g), dtype=F32), x, (q, s, z), g)
    # each group by itself, where the large ones do not hide the small
    for j in range(K // g):
        one = torch.zeros_like(x)
        one[:, j * g:(j + 1) * g] = x[:, j * g:(j + 1) * g]
        _close(dg.w4a16_linear_few(one, (q, s, z, g), dtype=F32), one, (q, s, z), g)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("max_tokens", [4, 20000])
def test_most_columns(max_tokens, dtype):
    V = 2**30 - 1
    x = torch.zeros((1, V), dtype=dtype, device="cuda")
    at = torch.tensor([0, 4097, V // 2, V - 3, V - 2, V - 1], device="cuda")
    x[0, at] = torch.tensor([1.0, 2.0, 4.0, 9.0, 16.0, 8.0], dtype=dtype, device="cuda")
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    tokens = torch.full((1, max_tokens), V - 1, dtype=torch.int32, device="cuda")
    tokens[0, :4] = i([V - 1, V, 2**31 - 1, -2**31])            # all but the first outside
    mask = torch.full((1, 2**25), -1, dtype=torch.int32, device="cuda")
    mask[0, -1] = ~(1 << 29)                                    # V - 2
    rules = dg.LogitRules(tokens=tokens, lengths=i([4]), presence=torch.tensor([2.0], device="cuda"),
                          bias_ids=i([[V - 3, V - 1]]), bias=torch.tensor([[-8.0, 4.0]], device="cuda"), mask=mask)
    y = dg.adjust_logits(x, rules, dtype=dtype)
    assert y[0, at].tolist() == [1.0, 2.0, 4.0, 1.0, -float("inf"), 10.0]
    assert int(torch.count_nonzero(y)) == 6
    _, smp, am = dg.sample_adjusted(x, rules, 5)
    assert int(am) == V - 1 and 0 <= int(smp) < V and int(smp) != V - 2
    dg.adjust_logits(x, rules, out=x)
    assert torch.equal(x.view(torch.int32 if dtype is F32 else torch.int16),
                       y.view(torch.int32 if dtype is F32 else torch.int16))


def test_highest_count():
    # one token 2^21 - 1 times, in the prompt too and with the last of 1023 biases
    L, V, n = 2**21 - 1, 5000, 1023
    tokens = torch.full((3, L), 4999, dtype=torch.int32)
    tokens[2] = torch.arange(L).remainder(3).int()
    ids = torch.full((3, n), 4999, dtype=torch.int32)
    u = dict(tokens=tokens, lengths=torch.full((3,), L, dtype=torch.int32),
             prompt_lengths=torch.tensor([0, 1, L // 2], dtype=torch.int32),
             repetition=torch.tensor([1.5, 1.1, 0.9]), frequency=torch.tensor([0.001, 1e-7, 0.01]),
             presence=torch.tensor([0.5, 0.25, 1.0]), bias_ids=ids,
             bias=torch.from_numpy(np.random.default_rng(1).standard_normal((3, n)).astype(np.float32)))
    l = torch.from_numpy(np.random.default_rng(2).standard_normal((3, V)).astype(np.float32))
    assert same_bits(dg.adjust_logits(l.cuda(), _dev(u)), torch.from_numpy(rules_ref.adjusted(l, u)))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_rules_and_logits_of_any_value(dtype):
    # zeros of both signs, subnormals, the ends of the type, infinities and NaN
    # under penalties, biases and scales of such values, bit for bit
    fi, inf, nan = torch.finfo(F32), float("inf"), float("nan")
    odd = [0.0, -0.0, 1.0, -1.5, 1e-40, -3e-45, fi.smallest_normal, 3e38, -3e38, inf, -inf, nan]
    rng = np.random.default_rng(7)
    t = torch.finfo(dtype)
    values = torch.tensor([0.0, -0.0, 1.0, -1.0, 1.7, -3.3, t.smallest_normal, -t.smallest_normal,
                           t.smallest_normal / 4, -t.smallest_normal / 2, t.max, t.min, inf, -inf, nan], dtype=dtype)
    R, V, L = 4 * len(odd), 1500, 400
    l = values[torch.from_numpy(rng.integers(0, len(values), (R, V)))]
    u = rules_ref.random_rules(rng, R, V, L=L, bias=30, mask=True)
    u["tokens"] = torch.from_numpy(rng.integers(0, V, (R, L)).astype(np.int32))
    for k, name in enumerate(("repetition", "frequency", "presence", "scale")):
        for i, v in enumerate(odd):
            u[name][k * len(odd) + i] = v
    u["bias"][:, 5:5 + len(odd)] = torch.tensor(odd)
    x = l.cuda()
    for drop in ((), ("scale",), ("repetition",), ("frequency",), ("presence",), ("bias", "bias_ids"), ("mask", "mask_row")):
        v = {k: a for k, a in u.items() if k not in drop}
        want = torch.from_numpy(rules_ref.adjusted(l, v))
        rules = _dev(v)
        assert same_bits(dg.adjust_logits(x, rules), want)
        y = x.clone()
        dg.adjust_logits(y, rules, out=y)
        assert same_bits(y, want.to(dtype))


@pytest.mark.parametrize("scale", [True, False])
@pytest.mark.parametrize("R,V,L", [(1000, 9000, 40), (1500, 20011, 17000)])
def test_in_place_in_a_graph(R, V, L, scale):
    # rows of shared sequences, several a workgroup; logits, lengths, sequences and
    # masks change between the replays
    rng = np.random.default_rng([R, scale])
    u = rules_ref.random_rules(rng, R, V, S=20, L=L, bias=3, mask=True, scale=scale)
    dev = {k: v.cuda() for k, v in u.items()}
    rules = dg.LogitRules(**dev)
    x = torch.empty((R, V), dtype=BF16, device="cuda")
    ws = torch.empty(dg.sample_adjusted_workspace_bytes(R, V), dtype=torch.uint8, device="cuda")
    x.normal_()
    dg.sample_adjusted(x, rules, 9, workspace=ws)
    dg.adjust_logits(x, rules, out=x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, smp, am = dg.sample_adjusted(x, rules, 9, workspace=ws)
        dg.adjust_logits(x, rules, out=x)
    for step in range(4):
        x.normal_()
        dev["lengths"].copy_(torch.randint(-1, L + 2, (20,)))
        dev["row_seq"].copy_(torch.randint(-1, 21, (R,)))
        dev["mask"].copy_(torch.randint(-2**31, 2**31, dev["mask"].shape))
        before = x.clone()
        graph.replay()
        want = rules_ref.adjusted(before.cpu(), {k: v.cpu() for k, v in dev.items()})
        assert same_bits(x, torch.from_numpy(want).to(BF16))
        rules_ref.check_sample(want, 9, None, smp, am)
        eager = dg.sample_adjusted(before, rules, 9)
        assert same_bits(h, eager[0]) and torch.equal(smp, eager[1]) and torch.equal(am, eager[2])
