"""GPU: the entropy of adjusted logits within the bound of its own roundings and sums
(tests/entropy_bound.py), from one logit to rows of many parts, flat and steep."""
import numpy as np
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import entropy_bound, rules_ref
from tests.test_gpu_logit_rules import CASES, TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    dg.lib()


def _dev(u):
    return dg.LogitRules(**{k: v.cuda() for k, v in u.items()})


@pytest.mark.parametrize("R,V,kw", CASES)
def test_entropy(R, V, kw):
    rng = np.random.default_rng([R, V, 2])
    for dtype in TYPES:
        l = torch.from_numpy((rng.standard_normal((R, V)) * 3).astype(np.float32)).to(dtype)
        u = rules_ref.random_rules(rng, R, V, **kw)
        h = dg.sample_adjusted(l.cuda(), _dev(u), draw=False)[0]
        entropy_bound.check(h, rules_ref.adjusted(l, u), kw.get("L", 50))


@pytest.mark.parametrize("spread", [0.0, 0.01, 30.0])
def test_entropy_of_flat_and_steep_rows(spread):
    rng = np.random.default_rng(3)
    l = (rng.standard_normal((3, 262144)) * spread).astype(np.float32)
    h = dg.sample_adjusted(torch.from_numpy(l).cuda(), dg.LogitRules(), draw=False)[0]
    entropy_bound.check(h, l, 0)
