"""Plain forms of the operators at the end of a step, for tests: the product
with 4-bit weights in 64 bits with the error its kernel may have, the rules on
logits with their stated fp32 roundings, and the sampler's outputs of adjusted
logits in 64 bits.

u32 = 2^-24 is half a step of fp32 (few_ref.U32).
"""
from __future__ import annotations

import numpy as np
import torch

import oracle
from tests.few_ref import U32

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half a step of the subnormals
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def codes(q):
    """uint8 [N, K/2] -> float64 [N, K]."""
    return np.stack((q & 15, q >> 4), axis=-1).reshape(q.shape[0], -1).astype(np.float64)


def linear(x, q, s, z, g, dtype):
    """y float64 [T, N] and the bound on an output of ``dtype``. x torch (CPU),
    q uint8, s and z fp16 (numpy, canonical).

    The kernel sums (16 + q) x and x over a group in fp32 (exact products),
    multiplies with s and s (16 + z) and adds groups and parts in fp32: each term's way
    has at most g additions in its group, 6 for products and the difference,
    and K / g + 16 to the end. Terms are at most |s| (31 + |16 + z|) |x|."""
    x = x.double().numpy()
    rep = lambda v: np.repeat(v.astype(np.float64), g, axis=1)
    w = (codes(q) - rep(z)) * rep(s)
    y = x @ w.T
    size = np.abs(x) @ (np.abs(rep(s)) * (31 + np.abs(16 + rep(z)))).T
    bound = 1.01 * U32 * (g + x.shape[1] / g + 22) * size
    return y, bound + HALF_STEP[dtype] * (np.abs(y) + bound) + TINY[dtype]


def adjusted(logits, rules, V=None):
    """The rules on logits (torch, CPU) as fp32 numpy [R, V], every operation
    rounded to fp32. ``rules``: LogitRules' arguments as CPU tensors."""
    u = {k: v.numpy() for k, v in rules.items()}
    l = logits.float().numpy().copy()
    R, V = l.shape
    f = np.float32
    S = next((len(u[k]) for k in ("lengths", "scale", "bias_ids") if k in u), 0)
    with np.errstate(all="ignore"):
        for r in range(R):
            s = int(u["row_seq"][r]) if "row_seq" in u else r
            if 0 <= s < S:
                if "tokens" in u:
                    L = u["tokens"].shape[1]
                    n = min(max(int(u["lengths"][s]), 0), L)
                    p = min(max(int(u["prompt_lengths"][s]), 0), n) if "prompt_lengths" in u else 0
                    tok = u["tokens"][s]
                    ok = lambda t: t[(t >= 0) & (t < V)]
                    seen = np.unique(ok(tok[:n]))
                    if "repetition" in u:
                        v = l[r, seen]
                        l[r, seen] = np.where(v > 0, v / u["repetition"][s], v * u["repetition"][s])
                    c = np.bincount(ok(tok[p:n]), minlength=V)[:V]
                    at = np.nonzero(c)[0]
                    if "frequency" in u:
                        l[r, at] = l[r, at] - u["frequency"][s] * c[at].astype(f)
                    if "presence" in u:
                        l[r, at] = l[r, at] - u["presence"][s]
                if "bias" in u:
                    last = {int(i): b for i, b in zip(u["bias_ids"][s], u["bias"][s]) if 0 <= i < V}
                    for i, b in last.items():
                        l[r, i] = l[r, i] + b
                if "scale" in u:
                    l[r] = l[r] * u["scale"][s]
            if "mask" in u:
                m = int(u["mask_row"][r]) if "mask_row" in u else r
                if 0 <= m < u["mask"].shape[0]:
                    bits = u["mask"][m].view(np.uint32)[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)
                    l[r, (bits & 1) == 0] = -np.inf
    assert l.dtype == f
    return l


def entropies(l):
    """Entropy float64 [R] of adjusted logits and the bound on its fp32 form.

    d = l - m is rounded once or twice, exp's argument and result as often: a
    relative error of at most 4 (1 + |d|) u32 for each exp. Sums have
    at most 64 terms one after the other in a lane and 40 joins, each with the
    partials' shift and scale (4 roundings): 230 u32. log z - s / z adds each
    part's own rounding. Together at most (240 + 4 (1 + |d|)) (1 + |d|) u32 p
    summed over the row, and 4 u32 (1 + log V)."""
    h, bound = np.zeros(len(l)), np.zeros(len(l))
    for r, row in enumerate(l.astype(np.float64)):
        v = row[row > -np.inf]
        if v.size == 0:
            continue
        d = v - v.max()
        e = np.exp(d)
        z = e.sum()
        h[r] = np.log(z) - (e * d).sum() / z
        one = 1 + np.abs(d)
        bound[r] = 1.01 * U32 * (((240 + 4 * one) * one * e).sum() / z + 4 * (1 + np.log(z)))
    return h, bound


def check_sample(l, seed, entropy, sample, argmax):
    """The sampler's outputs (torch, on any device) against adjusted logits l
    (fp32 numpy): argmax bit for bit; the sample the oracle's but where two
    scores lie within four steps of each other; entropy within its bound."""
    R, V = l.shape
    none = (l == -np.inf).all(1)
    am = argmax.cpu().numpy()
    assert np.array_equal(am, np.where(none, -1, l.argmax(1)))
    if entropy is not None:
        h, bound = entropies(l)
        err = np.abs(entropy.cpu().numpy().astype(np.float64) - h)
        assert (err <= bound).all(), (err / np.maximum(bound, 1e-30)).max()
    if sample is not None:
        smp = sample.cpu().numpy()
        assert np.array_equal(smp == -1, none)
        padded = np.full((R, (V + 3) // 4 * 4), -np.inf, dtype=np.float32)    # the oracle takes whole fours
        padded[:, :V] = l
        _, want, _, best = oracle.sample(padded, seed)
        for r in np.nonzero((smp != want) & ~none)[0]:
            got = oracle.gumbel_score(l[r, smp[r]], int(r), int(smp[r]), seed)
            assert abs(got - best[r]) <= 4 * np.spacing(np.float32(abs(best[r]))), (r, smp[r], want[r])


def random_rules(rng, R, V, S=None, L=50, bias=0, mask=False, scale=True, penalties=True, prompt=True):
    """Arguments of LogitRules as CPU tensors, with the edge values the rules
    allow: tokens and ids outside the vocabulary, lengths outside the buffer,
    rows without a sequence or a mask, a mask that leaves nothing."""
    t = torch.from_numpy
    u = {}
    own = S is None
    S = R if own else S
    f = lambda a: t(np.asarray(a, dtype=np.float32))
    i = lambda a: t(np.asarray(a, dtype=np.int32))
    if L:
        tok = np.minimum(rng.zipf(1.3, (S, L)) - 1, V + 3)
        tok[rng.random((S, L)) < 0.05] = -1
        u["tokens"] = i(tok)
        n = rng.integers(0, L + 1, S)
        n[0] = L + 5
        if S > 2:
            n[1], n[2] = 0, -3
        u["lengths"] = i(n)
        if prompt:
            p = (np.clip(n, 0, L) * rng.random(S)).astype(int)
            if S > 4:
                p[3], p[4] = L + 9, -2
            u["prompt_lengths"] = i(p)
        if penalties:
            u["repetition"] = f(rng.uniform(0.7, 1.6, S))
            u["frequency"] = f(rng.uniform(-0.3, 0.7, S))
            u["presence"] = f(rng.uniform(-0.3, 0.9, S))
    if bias:
        ids = rng.integers(-1, V + 1, (S, bias))
        if bias > 3:
            ids[:, 3] = ids[:, 1]                 # the same id twice: the last place counts
        u["bias_ids"], u["bias"] = i(ids), f(rng.standard_normal((S, bias)) * 3)
    if scale:
        u["scale"] = f(rng.uniform(0.5, 2.0, S))
    if not own:
        seq = rng.integers(0, S, R)
        if R > 3:
            seq[1], seq[2] = -1, S
        u["row_seq"] = i(seq)
    if mask:
        M = max(1, R // 2)
        m = rng.integers(0, 2 ** 32, (M, (V + 31) // 32), dtype=np.uint64).astype(np.uint32).view(np.int32)
        m[0] = 0
        if M > 1:
            m[1] = -1
        u["mask"] = t(m)
        u["mask_row"] = i(rng.integers(-1, M + 1, R))
        u["mask_row"][0] = 0
    return u
