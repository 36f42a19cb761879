"""GPU: the few-token operators together, as a serving step uses them: a
projection from activations, router logits from 8-bit codes, the routed experts,
the LM head's logits and the sampler. Each step's output is held against its own
definition on the inputs it was given, the whole chain against its parts, its
replays in a graph and its runs on other streams."""
import numpy as np
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import few_ref

pytestmark = pytest.mark.gpu

D, M, E, TOPK, V = 512, 192, 12, 3, 4096


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    dg.lib()


class Model:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, device="cuda", generator=g) * 0.05
        self.proj = dg.quantize_rows_i8(rnd(D, D))
        self.route = dg.quantize_rows_i8(rnd(E, D) * 20)
        self.head = dg.quantize_rows_i8(rnd(V, D))
        self.gu = dg.pack_tiled((*dg.quantize_rtn(rnd(E, 2 * M, D), 128), 128))
        self.dn = dg.pack_tiled((*dg.quantize_rtn(rnd(E, D, M), 64), 64))

    def buffers(self, T):
        byte = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        few = dg.moe_few_workspace_bytes(T, TOPK, E, D, M, self.gu[3], self.dn[3])
        return dict(tok=byte(dg.w8a8_workspace_bytes(T, D)), few=byte(few))

    def step(self, x, buf, seed=5):
        h = dg.w8a8_linear_tokens(x, self.proj, dtype=torch.float16, workspace=buf["tok"])
        q, s = dg.quantize_rows_i8(h)
        lg = dg.w8a8_linear(q, s, self.route, dtype=torch.float32)
        y = dg.moe_few_routed(h, lg, TOPK, self.gu, self.dn, workspace=buf["few"])
        logits = dg.w8a8_linear_tokens(y, self.head, dtype=torch.float32, workspace=buf["tok"])
        _, smp, am = dg.sample(logits, seed)
        return h, lg, y, logits, smp, am


def _x(T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, D), device="cuda", generator=g).to(torch.bfloat16)


def _same(a, b):
    return all(few_ref.same_bits(u, v) if u.is_floating_point() else torch.equal(u.cpu(), v.cpu())
               for u, v in zip(a, b))


@pytest.mark.parametrize("T", [1, 5, 30])
def test_step_by_step(T):
    m = Model()
    x = _x(T, T)
    h, lg, y, logits, smp, am = m.step(x, m.buffers(T))
    host = lambda w: (w[0].cpu().numpy(), w[1].cpu().numpy())
    q, s = few_ref.quantize_rows(x.cpu())
    assert few_ref.same_bits(h, few_ref.product(q, s, *host(m.proj), torch.float16))
    q, s = few_ref.quantize_rows(h.cpu())
    assert few_ref.same_bits(lg, few_ref.product(q, s, *host(m.route), torch.float32))
    ids, w = dg.router(lg, TOPK)
    assert few_ref.same_bits(y, dg.moe_few(h, ids, w, m.gu, m.dn))
    q, s = few_ref.quantize_rows(y.cpu())
    ref = few_ref.product(q, s, *host(m.head), torch.float32)
    assert few_ref.same_bits(logits, ref)
    assert torch.equal(am.cpu().long(), ref.argmax(1))
    # each token's results are its own: a batch gives what its tokens give alone
    for t in {0, T - 1}:
        alone = m.step(x[t:t + 1].contiguous(), m.buffers(1))
        assert few_ref.same_bits(alone[0], h[t:t + 1]) and few_ref.same_bits(alone[1], lg[t:t + 1])


@pytest.mark.parametrize("T", [1, 5, 30])
def test_step_captured(T):
    m = Model()
    x = _x(T, 1).clone()
    buf, other = m.buffers(T), m.buffers(T)
    m.step(x, buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = m.step(x, buf)
    for i in range(4):
        x.copy_(_x(T, 10 + i))
        graph.replay()
        eager = m.step(x, other)
        torch.cuda.synchronize()
        assert _same(outs, eager), i


def test_steps_on_two_streams():
    m = Model()
    xs = [_x(6, 1), _x(20, 2)]
    want = [m.step(x, m.buffers(x.shape[0])) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    bufs = [m.buffers(x.shape[0]) for x in xs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = m.step(xs[i], bufs[i])
    torch.cuda.synchronize()
    assert _same(got[0], want[0]) and _same(got[1], want[1])


def test_empty_workspace():
    # a workspace without bytes is an error, not the size query that a NULL one
    # is in the C ABI; for no tokens it is enough
    m = Model()
    x = torch.randn((2, D), device="cuda").half()
    lg = torch.randn((2, E), device="cuda")
    ids, w = dg.router(lg, TOPK)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    calls = [lambda n: dg.w8a8_linear_tokens(x[:n], m.proj, workspace=none),
             lambda n: dg.moe_few(x[:n], ids[:n], w[:n], m.gu, m.dn, workspace=none),
             lambda n: dg.moe_few_routed(x[:n], lg[:n], TOPK, m.gu, m.dn, workspace=none)]
    for call in calls:
        with pytest.raises(ValueError, match="workspace"):
            call(2)
        assert call(0).shape == (0, D)
