"""GPU: calls of the rules on logits and of the sampler with them beside each other,
each call's outputs looked at."""
import threading

import numpy as np
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import rules_ref
from tests.few_ref import same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    dg.lib()


def _dev(u):
    return dg.LogitRules(**{k: v.cuda() for k, v in u.items()})


def test_two_host_threads_call_by_call():
    # every call's outputs, on streams of their own, with the same rules object: a
    # batch whose workspace two calls at once must not share, and another one
    rng = np.random.default_rng(16)
    batches = []
    for R, V in ((8, 30000), (5, 90000)):
        u = rules_ref.random_rules(rng, R, V, L=200, bias=3, mask=True)
        x = torch.from_numpy((rng.standard_normal((R, V)) * 3).astype(np.float32)).cuda()
        rules = _dev(u)
        batches.append((x, rules, [dg.sample_adjusted(x, rules, s) for s in range(4)], dg.adjust_logits(x, rules)))
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got = []
                for i in range(20):
                    for x, rules, _, _ in batches:
                        got.append((*dg.sample_adjusted(x, rules, i % 4), dg.adjust_logits(x, rules)))
                torch.cuda.current_stream().synchronize()
                for i in range(20):
                    for k, (_, _, want, adj) in enumerate(batches):
                        h, smp, am, a = got[2 * i + k]
                        w = want[i % 4]
                        if not (same_bits(h, w[0]) and torch.equal(smp, w[1]) and torch.equal(am, w[2])
                                and same_bits(a, adj)):
                            bad.append((i, k))
        except Exception as e:
            bad.append(e)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("R,V,S", [(3, 5000, 3), (40, 70000, 40), (1500, 9000, 7)])
def test_a_larger_buffer_changes_nothing(R, V, S):
    # the same tokens in a buffer of long contexts, and in a view of its columns in use
    rng = np.random.default_rng(V)
    u = {k: v.cuda() for k, v in rules_ref.random_rules(rng, R, V, S=S, L=300, bias=4).items()}
    u["lengths"].clamp_(max=300)
    x = torch.from_numpy((rng.standard_normal((R, V)) * 3).astype(np.float32)).cuda()
    wide = torch.full((S, 40000), 7, dtype=torch.int32, device="cuda")
    wide[:, :300] = u["tokens"]
    want = None
    for tokens in (u["tokens"], wide[:, :300], wide):
        rules = dg.LogitRules(**{**u, "tokens": tokens})
        got = (*dg.sample_adjusted(x, rules, 8), dg.adjust_logits(x, rules))
        want = want or got
        assert same_bits(got[0], want[0]) and same_bits(got[3], want[3])
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
