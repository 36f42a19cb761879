"""GPU: the operators at the end of a serving step together, as a loop uses
them: the LM head on 4-bit weights, the requests' rules, the draw, the drawn
tokens appended to their sequences. Each step is held against its parts'
definitions, and the loop captured into a graph against the eager one."""
import numpy as np
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import rules_ref
from tests.few_ref import same_bits

pytestmark = pytest.mark.gpu

D, V, L = 512, 3001, 40


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    dg.lib()


class Loop:
    """T sequences, a prompt of a few tokens each, their hidden states a fixed
    table by token and their rules."""

    def __init__(self, T, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, device="cuda", generator=g)
        self.T = T
        self.table = (rnd(V, D) * 0.7).to(torch.bfloat16)
        self.head = (*dg.quantize_rtn(rnd(V, D) * 0.05, 128), 128)
        self.tokens = torch.randint(0, V, (T, L), device="cuda", dtype=torch.int32, generator=g)
        self.lengths = torch.randint(1, 6, (T,), device="cuda", dtype=torch.int32, generator=g)
        self.u = dict(tokens=self.tokens, lengths=self.lengths, prompt_lengths=self.lengths.clone(),
                      repetition=1.1 + 0.2 * torch.rand(T, device="cuda", generator=g),
                      frequency=0.3 * torch.rand(T, device="cuda", generator=g),
                      presence=0.3 * torch.rand(T, device="cuda", generator=g),
                      scale=1 / (0.6 + torch.rand(T, device="cuda", generator=g)),
                      bias_ids=torch.randint(-1, V, (T, 5), device="cuda", dtype=torch.int32, generator=g),
                      bias=rnd(T, 5),
                      mask=torch.randint(-2**31, 2**31, (T, (V + 31) // 32), device="cuda", generator=g).int(),
                      mask_row=torch.arange(T, device="cuda", dtype=torch.int32) % 2 * 2 - 1)
        self.rules = dg.LogitRules(**self.u)
        self.x = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
        self.logits = torch.empty((T, V), device="cuda")
        self.ws = torch.empty(dg.sample_adjusted_workspace_bytes(T, V), dtype=torch.uint8, device="cuda")

    def step(self, seed=3):
        last = self.tokens.gather(1, (self.lengths - 1).long()[:, None])
        torch.index_select(self.table, 0, last[:, 0], out=self.x)
        dg.w4a16_linear_few(self.x, self.head, out=self.logits)
        h, smp, am = dg.sample_adjusted(self.logits, self.rules, seed, workspace=self.ws)
        self.tokens.scatter_(1, self.lengths.long()[:, None], smp[:, None])
        self.lengths += 1
        return h, smp, am


@pytest.mark.parametrize("T", [1, 6, 33])
def test_step_by_step(T):
    m = Loop(T)
    host = [v.cpu().numpy() for v in m.head[:3]]
    for i in range(4):
        u = {k: v.cpu().clone() for k, v in m.u.items()}
        h, smp, am = m.step(seed=i)
        want, bound = rules_ref.linear(m.x.cpu(), *host, 128, torch.float32)
        assert (np.abs(m.logits.cpu().double().numpy() - want) <= bound).all()
        l = rules_ref.adjusted(m.logits.cpu(), u)
        rules_ref.check_sample(l, i, h, smp, am)
        assert same_bits(dg.adjust_logits(m.logits, dg.LogitRules(**{k: v.cuda() for k, v in u.items()})),
                         torch.from_numpy(l))
        at = u["lengths"].long()
        assert torch.equal(m.tokens.cpu().gather(1, at[:, None])[:, 0], smp.cpu())


@pytest.mark.parametrize("T", [1, 17])
def test_captured(T):
    a, b = Loop(T), Loop(T)
    tokens, lengths = a.tokens.clone(), a.lengths.clone()
    a.step()
    torch.cuda.synchronize()
    a.tokens.copy_(tokens)
    a.lengths.copy_(lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = a.step()
    a.tokens.copy_(tokens)
    a.lengths.copy_(lengths)
    for i in range(6):
        graph.replay()
        want = b.step()
        torch.cuda.synchronize()
        assert same_bits(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2]), i
        assert torch.equal(a.tokens, b.tokens) and torch.equal(a.lengths, b.lengths)


def test_two_batches_on_two_streams():
    loops, alone = [Loop(5, 1), Loop(12, 2)], [Loop(5, 1), Loop(12, 2)]
    want = [[m.step(i) for i in range(5)] for m in alone]
    streams = [torch.cuda.Stream() for _ in loops]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(loops[k].step(i))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for x, y in zip(g, w):
            assert same_bits(x[0], y[0]) and torch.equal(x[1], y[1]) and torch.equal(x[2], y[2])
