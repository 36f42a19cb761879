"""GPU: a batch's rules on its logits, bit for bit against their stated fp32
roundings, and the sampler on adjusted logits against those and the oracle
(tests/rules_ref.py)."""
import numpy as np
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import rules_ref
from tests.few_ref import same_bits

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    dg.lib()


def _logits(rng, R, V, dtype, inf=0.0):
    l = torch.from_numpy((rng.standard_normal((R, V)) * 3).astype(np.float32))
    if inf:
        l[torch.from_numpy(rng.random((R, V)) < inf)] = float("-inf")
    return l.to(dtype)


def _rules(u):
    return dg.LogitRules(**{k: v.cuda() for k, v in u.items()})


def _case(rng, R, V, dtype, inf=0.0, **kw):
    l = _logits(rng, R, V, dtype, inf)
    u = rules_ref.random_rules(rng, R, V, **kw)
    return l, u, _rules(u)


CASES = [
    (1, 1, dict(L=3)), (1, 5, dict(L=1, bias=2)), (2, 31, dict(L=40, bias=5, mask=True)), (3, 33, dict(L=0, mask=True)),
    (5, 1000, dict(L=700, bias=40, mask=True)), (1, 32000, dict(L=300)), (4, 2048, dict(L=50, bias=1)),
    (7, 4097, dict(L=5000, S=3, mask=True)), (33, 8191, dict(L=64, bias=1023)), (2, 100003, dict(L=30000, bias=300, S=1)),
    (64, 6000, dict(L=20, S=2, scale=False)), (9, 515, dict(L=0, bias=12, penalties=False)),
    (6, 3000, dict(L=90, prompt=False, mask=True)), (3, 20000, dict(L=0, scale=False, mask=True)),
    (300, 1027, dict(L=33, S=7, bias=3, mask=True)), (5, 262144, dict(L=2000, mask=True, bias=9)),
    (40, 70000, dict(L=400, S=5)), (130, 33000, dict(L=90, mask=True, S=130)), (64, 70001, dict(L=17000, bias=2, S=9)),
]


@pytest.mark.parametrize("R,V,kw", CASES)
def test_adjust(R, V, kw):
    rng = np.random.default_rng([R, V])
    for dtype in TYPES:
        l, u, rules = _case(rng, R, V, dtype, inf=0.01, **kw)
        want = torch.from_numpy(rules_ref.adjusted(l, u))
        x = l.cuda()
        assert same_bits(dg.adjust_logits(x, rules), want)
        own = dg.adjust_logits(x, rules, dtype=dtype)
        assert own.dtype == dtype and same_bits(own, want.to(dtype))
        assert same_bits(x, l)
        assert dg.adjust_logits(x, rules, out=x) is x
        assert same_bits(x, want.to(dtype))


@pytest.mark.parametrize("R,V,kw", CASES)
def test_sample(R, V, kw):
    rng = np.random.default_rng([R, V, 1])
    for dtype in TYPES:
        l, u, rules = _case(rng, R, V, dtype, inf=0.01, **kw)
        x = l.cuda()
        seed = int(rng.integers(2 ** 63))
        h, smp, am = dg.sample_adjusted(x, rules, seed)
        rules_ref.check_sample(rules_ref.adjusted(l, u), seed, h, smp, am)
        assert same_bits(x, l)
        # any of the outputs alone, and the call again: the same bits
        h2, none, am2 = dg.sample_adjusted(x, rules, seed, draw=False)
        none2, smp2, am3 = dg.sample_adjusted(x, rules, seed, entropy=False)
        assert none is None and none2 is None
        assert same_bits(h, h2) and torch.equal(smp, smp2) and torch.equal(am, am2) and torch.equal(am, am3)


@pytest.mark.parametrize("V", [9000, 20011])
def test_columns_with_words_from_few_to_all(V):
    # runs of n tokens' columns, scattered and side by side, so that waves have
    # none, few, as many as their lanes take in turns, more than that, and all;
    # then rows that share those sequences, in any order
    runs = [0, 1, 63, 64, 65, 127, 128, 129, 130, 500, 1024, V]
    L = max(runs)
    rng = np.random.default_rng(V)
    S = 2 * len(runs)
    u = rules_ref.random_rules(rng, S, V, L=L, bias=7)
    for i, n in enumerate(runs):
        u["tokens"][2 * i, :n] = torch.from_numpy(rng.permutation(min(1024, V))[:n] if n <= 1024
                                                  else rng.permutation(V)).int()
        u["tokens"][2 * i + 1, :n] = torch.arange(n).int()
        u["lengths"][2 * i:2 * i + 2] = n
    u["prompt_lengths"] = u["lengths"] // 2
    for R in (S, 400):
        u["row_seq"] = torch.from_numpy(np.sort(rng.integers(0, S, R)) if R != S else rng.permutation(S)).int()
        for dtype in TYPES:
            l = _logits(rng, R, V, dtype, inf=0.01)
            rules, want, x = _rules(u), rules_ref.adjusted(l, u), l.cuda()
            assert same_bits(dg.adjust_logits(x, rules), torch.from_numpy(want))
            rules_ref.check_sample(want, R, *dg.sample_adjusted(x, rules, R))
            plain = {k: v for k, v in u.items() if k != "scale"}
            dg.adjust_logits(x, _rules(plain), out=x)
            assert same_bits(x, torch.from_numpy(rules_ref.adjusted(l, plain)).to(dtype))


def test_no_rules():
    # nothing but a copy, and dgw4_sample's own draws
    rng = np.random.default_rng(0)
    x = _logits(rng, 12, 5000, F32).cuda()
    rules = dg.LogitRules()
    assert same_bits(dg.adjust_logits(x, rules), x)
    h, smp, am = dg.sample_adjusted(x, rules, 99)
    h0, smp0, am0 = dg.sample(x, 99)
    assert torch.equal(smp, smp0) and torch.equal(am, am0)
    assert (h - h0).abs().max() < 1e-5 * h0.abs().max()
    y = _logits(rng, 12, 4999, BF16).cuda()
    assert same_bits(dg.adjust_logits(y, rules), y.float())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_masked_places_hold_anything(dtype):
    # NaN and infinities where the mask does not allow a token, the type's
    # lowest value as a mask of its own, rows with one and no token left
    rng = np.random.default_rng(5)
    R, V = 6, 3001
    l = _logits(rng, R, V, dtype)
    mask = torch.from_numpy(rng.integers(-2**31, 2**31, (R, (V + 31) // 32)).astype(np.int32))
    mask[4] = 0
    mask[5] = 0
    mask[5, 17] = 1 << 5
    bits = (mask.numpy().view(np.uint32)[:, np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
    out = np.argwhere(bits == 0)
    for k, v in enumerate((float("nan"), float("inf"), float("-inf"), torch.finfo(dtype).max)):
        for r, c in out[k::7]:
            l[r, c] = v
    l[0, :1000] = torch.finfo(dtype).min
    u = dict(mask=mask, tokens=torch.from_numpy(rng.integers(0, V, (R, 500)).astype(np.int32)),
             lengths=torch.full((R,), 500, dtype=torch.int32), repetition=torch.full((R,), 1.25))
    rules = _rules(u)
    want = rules_ref.adjusted(l, u)
    assert not np.isnan(want).any()
    assert same_bits(dg.adjust_logits(l.cuda(), rules), torch.from_numpy(want))
    h, smp, am = dg.sample_adjusted(l.cuda(), rules, 3)
    rules_ref.check_sample(want, 3, h, smp, am)
    assert h[4] == 0 and smp[4] == -1 and am[4] == -1
    assert h[5] == 0 and smp[5] == 17 * 32 + 5 and am[5] == 17 * 32 + 5


def test_ties():
    # equal logits across lanes, waves and workgroups: the lowest token wins,
    # also where a penalty makes them equal
    V = 60000
    rng = np.random.default_rng(8)
    for at in ([5, 6], [100, 59999], [2047, 2048], [31, 40000], [1023, 1024, 4096]):
        l = _logits(rng, 3, V, F32).clamp_(max=8)
        l[:, at] = 9.0
        l[1, at[0]] = 10.0
        u = dict(tokens=torch.tensor([[0], [at[0]], [at[0]]], dtype=torch.int32),
                 lengths=torch.tensor([1, 1, 1], dtype=torch.int32), presence=torch.tensor([0.0, 1.0, 0.5]))
        am = dg.sample_adjusted(l.cuda(), _rules(u), 1)[2]
        assert am.tolist() == [at[0], at[0], at[1]]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_strided(dtype):
    # rows apart and from odd elements on, of logits, output and rules
    rng = np.random.default_rng(11)
    R, V = 9, 2050
    l, u, _ = _case(rng, R, V, dtype, L=60, bias=7, mask=True)
    wide = torch.zeros((R + 1, V + 13), dtype=dtype, device="cuda")
    x = wide[1:, 3:V + 3]
    x.copy_(l)
    dev = {k: v.cuda() for k, v in u.items()}
    for k in ("tokens", "bias_ids", "bias", "mask"):
        w = torch.full((dev[k].shape[0], dev[k].shape[1] + 11), 1, dtype=dev[k].dtype, device="cuda")
        w[:, 5:5 + dev[k].shape[1]] = dev[k]
        dev[k] = w[:, 5:5 + dev[k].shape[1]]
    rules = dg.LogitRules(**dev)
    want = torch.from_numpy(rules_ref.adjusted(l, u))
    buf = torch.full((R + 2, V + 5), 6.0, device="cuda")
    dg.adjust_logits(x, rules, out=buf[1:R + 1, 1:V + 1])
    assert same_bits(buf[1:R + 1, 1:V + 1], want)
    buf[1:R + 1, 1:V + 1] = 6.0
    assert (buf == 6.0).all()
    h, smp, am = dg.sample_adjusted(x, rules, 4)
    rules_ref.check_sample(want.numpy(), 4, h, smp, am)
    before = wide.clone()
    dg.adjust_logits(x, rules, out=x)
    assert same_bits(x, want.to(dtype))
    before[1:, 3:V + 3] = x
    assert same_bits(wide, before)


def test_interleaved_output():
    # the output's rows between those of the logits
    rng = np.random.default_rng(12)
    l, u, rules = _case(rng, 7, 700, F32, L=20)
    buf = torch.zeros((7, 1400), device="cuda")
    buf[:, :700] = l.cuda()
    dg.adjust_logits(buf[:, :700], rules, out=buf[:, 700:])
    assert same_bits(buf[:, 700:], torch.from_numpy(rules_ref.adjusted(l, u))) and same_bits(buf[:, :700], l)
    with pytest.raises(dg.Dgw4Error, match="INVALID"):
        dg.adjust_logits(buf[:, :700], rules, out=buf[:, 699:1399])


def test_many_rows():
    # more rows than a grid's second dimension takes
    rng = np.random.default_rng(13)
    R, V = 70001, 40
    l, u, rules = _case(rng, R, V, F16, S=3, L=9)
    want = rules_ref.adjusted(l, u)
    assert same_bits(dg.adjust_logits(l.cuda(), rules), torch.from_numpy(want))
    am = dg.sample_adjusted(l.cuda(), rules, 1, draw=False)[2]
    assert np.array_equal(am.cpu().numpy(), want.argmax(1))


def test_offsets_past_32_bits():
    # more logits than 32 bits count, tokens at the end of long rows
    R, V = 9, 1 << 28
    x = torch.zeros((R, V), dtype=F16, device="cuda")
    at = torch.tensor([0, 1, V // 2 + 3, V - 2, V - 1], device="cuda")
    x[:, at] = torch.tensor([1.0, 2.0, 4.0, 3.0, 8.0], dtype=F16, device="cuda")
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    rules = dg.LogitRules(tokens=i([[V - 1, V - 1, V - 2]]).expand(R, 3).contiguous(), lengths=i([3] * R),
                          presence=torch.full((R,), 1.0, device="cuda"),
                          frequency=torch.full((R,), 2.0, device="cuda"))
    out = dg.adjust_logits(x, rules, dtype=F16)
    assert (out[:, at].float() == torch.tensor([1.0, 2.0, 4.0, 0.0, 3.0], device="cuda")).all()
    assert int(torch.count_nonzero(out[R - 1])) == 4
    h, _, am = dg.sample_adjusted(x, rules, draw=False)
    assert (am == V // 2 + 3).all()
    # Nearly all of the weight is on the zeros. A row has 2^18 parts, 1024 one after
    # the other in a thread of the join: z and s are off by at most 1324 u32 of
    # themselves, and |s / z| is below 9.
    z = V - 4 + sum(np.exp([1.0, 2.0, 4.0, 3.0]))
    want = np.log(z) - sum(v * np.exp(v) for v in (1.0, 2.0, 4.0, 3.0)) / z
    assert np.abs(h.cpu().numpy() - want).max() <= 1.01 * (1 + 2 * 9) * 1324 * 2.0 ** -24


def test_two_host_threads():
    # two threads on streams of their own, the same rules object
    import threading
    rng = np.random.default_rng(16)
    l, u, rules = _case(rng, 8, 30000, F32, L=200, bias=3, mask=True)
    x = l.cuda()
    want = dg.sample_adjusted(x, rules, 5)
    adj = dg.adjust_logits(x, rules)
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got, a = dg.sample_adjusted(x, rules, 5), dg.adjust_logits(x, rules)
                torch.cuda.current_stream().synchronize()
                if not (same_bits(got[0], want[0]) and torch.equal(got[1], want[1]) and same_bits(a, adj)):
                    bad.append("differs")
        except Exception as e:
            bad.append(e)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_two_graphs_share_a_workspace():
    # replayed one after the other on one stream
    rng = np.random.default_rng(17)
    cases = [_case(rng, R, V, F32, L=60, mask=True) for R, V in ((6, 50000), (2, 200000))]
    n = max(dg.sample_adjusted_workspace_bytes(*c[0].shape) for c in cases)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    xs = [c[0].cuda() for c in cases]
    for x, c in zip(xs, cases):
        dg.sample_adjusted(x, c[2], 7, workspace=ws)
    torch.cuda.synchronize()
    graphs, got = [], []
    for x, c in zip(xs, cases):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(dg.sample_adjusted(x, c[2], 7, workspace=ws))
    for _ in range(3):
        for g in graphs:
            g.replay()
        for k, (l, u, _) in enumerate(cases):
            rules_ref.check_sample(rules_ref.adjusted(l, u), 7, *got[k])


def test_counts():
    # one token very often, in the prompt and after it
    L, V = 100000, 5000
    tok = torch.full((2, L), 17, dtype=torch.int32)
    tok[1, ::2] = 4095
    u = dict(tokens=tok, lengths=torch.tensor([L, L], dtype=torch.int32),
             prompt_lengths=torch.tensor([1, 50001], dtype=torch.int32), repetition=torch.tensor([1.5, 1.1]),
             frequency=torch.tensor([0.001, 0.01]), presence=torch.tensor([0.5, 0.25]))
    l = _logits(np.random.default_rng(1), 2, V, F32)
    assert same_bits(dg.adjust_logits(l.cuda(), _rules(u)), torch.from_numpy(rules_ref.adjusted(l, u)))


def test_rules_change_in_place():
    # a step appends its tokens and moves the lengths on: the same rules object
    rng = np.random.default_rng(14)
    R, V, L = 4, 900, 30
    l = _logits(rng, R, V, F32)
    u = dict(tokens=torch.zeros((R, L), dtype=torch.int32), lengths=torch.zeros(R, dtype=torch.int32),
             prompt_lengths=torch.zeros(R, dtype=torch.int32), repetition=torch.full((R,), 1.3),
             frequency=torch.full((R,), 0.4), presence=torch.full((R,), 0.2))
    dev = {k: v.cuda() for k, v in u.items()}
    rules, x = dg.LogitRules(**dev), l.cuda()
    for step in range(6):
        want = rules_ref.adjusted(l, u)
        h, smp, am = dg.sample_adjusted(x, rules, step)
        rules_ref.check_sample(want, step, h, smp, am)
        dev["tokens"][:, step] = smp
        dev["lengths"] += 1
        u["tokens"][:, step] = smp.cpu()
        u["lengths"] += 1


def test_graph_and_streams():
    rng = np.random.default_rng(15)
    R, V = 5, 40000
    l, u, rules = _case(rng, R, V, BF16, L=300, bias=4, mask=True)
    x = l.cuda()
    ws = torch.empty(dg.sample_adjusted_workspace_bytes(R, V), dtype=torch.uint8, device="cuda")
    adj = torch.empty((R, V), device="cuda")
    dg.sample_adjusted(x, rules, 5, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dg.sample_adjusted(x, rules, 5, workspace=ws)
        dg.adjust_logits(x, rules, out=adj)
    for i in range(4):
        x.copy_(_logits(rng, R, V, BF16))
        graph.replay()
        eager = dg.sample_adjusted(x, rules, 5)
        assert same_bits(got[0], eager[0]) and torch.equal(got[1], eager[1]) and torch.equal(got[2], eager[2])
        assert same_bits(adj, dg.adjust_logits(x, rules))
    xs = [_logits(rng, R, V, F32).cuda() for _ in range(2)]
    want = [dg.sample_adjusted(v, rules, 6) for v in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        out = []
        for v, st in zip(xs, streams):
            with torch.cuda.stream(st):
                out.append(dg.sample_adjusted(v, rules, 6))
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert same_bits(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


def test_refusals():
    x = torch.zeros((4, 100), device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.zeros(s, device="cuda")
    for kw in (dict(tokens=i(4, 5)), dict(lengths=i(4)), dict(repetition=f(4)), dict(prompt_lengths=i(4)),
               dict(bias=f(4, 2)), dict(bias_ids=i(4, 2)), dict(mask_row=i(4)),
               dict(tokens=i(4, 5), lengths=i(3)), dict(tokens=i(4, 0), lengths=i(4)),
               dict(tokens=i(4, 5), lengths=i(4), presence=f(5)), dict(bias_ids=i(4, 2), bias=f(4, 3)),
               dict(bias_ids=i(4, 9)[:, :2], bias=f(4, 2)), dict(scale=f(4, 1)),
               dict(scale=f(4), bias_ids=i(3, 2), bias=f(3, 2)), dict(scale=f(8)[::2])):
        with pytest.raises(ValueError):
            dg.LogitRules(**kw)
    for kw in (dict(tokens=f(4, 5), lengths=i(4)), dict(scale=i(4)), dict(mask=f(4, 4)), dict(row_seq=f(4))):
        with pytest.raises(TypeError):
            dg.LogitRules(**kw)
    for kw in (dict(scale=f(3)), dict(scale=f(1), row_seq=i(3)), dict(mask=i(4, 3)), dict(mask=i(3, 4)),
               dict(mask=i(2, 4), mask_row=i(3))):
        rules = dg.LogitRules(**kw)
        with pytest.raises(ValueError):
            dg.adjust_logits(x, rules)
        with pytest.raises(ValueError):
            dg.sample_adjusted(x, rules)
    none = dg.LogitRules()
    with pytest.raises(TypeError):
        dg.adjust_logits(x, dict())
    with pytest.raises(TypeError):
        dg.adjust_logits(x.double(), none)
    with pytest.raises(dg.Dgw4Error, match="UNSUPPORTED"):
        dg.adjust_logits(x, none, dtype=F16)
    with pytest.raises(ValueError, match="out"):
        dg.adjust_logits(x, none, out=f(4, 99))
    with pytest.raises(ValueError, match="workspace"):
        dg.sample_adjusted(x, none, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(dg.Dgw4Error, match="WORKSPACE"):
        dg.sample_adjusted(x, none, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert dg.adjust_logits(x[:0], none).shape == (0, 100)
    assert dg.sample_adjusted(x[:0], none)[2].shape == (0,)


def test_as_many_rows_as_an_int_counts():
    """2^31 - 1 rows of one column: the last rows are changed as the others."""
    R = 2**31 - 1
    x = torch.empty(R, 1, device="cuda", dtype=torch.float16)
    at = x.view(-1)
    at.fill_(1.0)
    ends = torch.arange(-2000, 2000, device="cuda")
    at[ends] = (ends % 2000).to(torch.float16)
    y = dg.adjust_logits(x, dg.LogitRules(), dtype=torch.float16)
    assert torch.equal(y, x)
