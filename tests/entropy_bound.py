"""How far the sampler's entropy of adjusted logits may be off, by its roundings and
the way its sums are cut up (test helper).

u = 2^-24 is half a step of fp32, D = max - l of a logit, p its probability, z the
sum of exp(-D), H1 the sum of p D; the entropy is log z + H1.

Each logit's exp is taken in two pieces (against its part's maximum, then the part's
against the row's), whose distances add up to D: rounding them, the product with
log2 e and that constant, 3 D u; the hardware's exp2, 2 u each; the product of the
pieces, u. Additions on a term's way: E in a lane, 6 across a wave, as many as a
thread of the join has parts, 6 and 2 to the end. So a term of z is off by at most
(n + 5 + 3 D) u of itself, n = E + 14 + ceil(parts / 256). A term of the sum of p D
takes four more: its distance, its product and the two of a part's shift. The
logarithm, its constant, the quotient and the difference: 6 (1 + log z) + 3 H1.
"""
from __future__ import annotations

import numpy as np

from tests.few_ref import U32

LONG = 16384                 # tokens of a buffer from which a workgroup has 512 threads, not 256


def cut(R, V, max_tokens):
    """(columns of a thread, parts of a row)."""
    e = 16 if R * (-(-V // 1024)) >= 4096 else 8
    threads = 512 if max_tokens >= LONG else 256
    return e, -(-V // (threads * e)) * (threads // 64)


def check(entropy, l, max_tokens):
    """entropy (torch, on any device) against adjusted logits l (fp32 numpy [R, V])."""
    e, parts = cut(*l.shape, max_tokens)
    n = e + 14 + -(-parts // 256)
    got = entropy.cpu().numpy().astype(np.float64)
    for r, row in enumerate(l):
        v = row[row > -np.inf].astype(np.float64)
        if v.size == 0:
            assert got[r] == 0
            continue
        d = v.max() - v
        p = np.exp(-d)
        z = p.sum()
        p /= z
        h1 = (p * d).sum()
        a = (p * (n + 5 + 3 * d)).sum()
        b = (p * d * (n + 9 + 3 * d)).sum()
        bound = 1.01 * U32 * ((1 + h1) * a + b + 6 * (1 + np.log(z)) + 3 * h1)
        assert abs(got[r] - (np.log(z) + h1)) <= bound, (r, got[r], np.log(z) + h1, bound)
