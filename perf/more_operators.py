"""The end of a serving step at few tokens, as measured cases.

A step ends with the LM head and the choice of the next tokens. Its dense
products run on the same 4-bit weights as the experts, for one to a few dozen
tokens; each sequence's logits are then changed by the request's rules and
sampled:

* ``linear``  the product of a few tokens with 4-bit weights (codes, group
              scales, group zero points), any channels, fp16 / bf16 in,
              fp16 / bf16 / fp32 out;
* ``adjust``  a request's rules on its logits: penalties for the tokens that
              its sequence holds, biases, a scale (one over a temperature), a
              grammar's mask of allowed tokens;
* ``sample``  the same rules inside the sampler's one pass over the logits:
              entropy, Gumbel-max sample and argmax of the adjusted logits.

The rules, for logit l of token v in a row of sequence s, in this order:
seen anywhere in the sequence: l / repetition (l > 0) or l * repetition; c
times among the generated tokens, c > 0: l - frequency * c, then l - presence;
l + bias of v; l * scale; -inf where the row's mask does not allow v.

``own`` false: plain elementary torch operations in 32 bits. ``own`` true:
the calls a user makes of ``w4a16_grouped_moe_amd``. ``exact`` computes the
definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}

# The largest work of a listed case, which drawn ones stay below.
MAX_WEIGHT = 262144 * 2816
MAX_LOGITS = 256 * 262144

# Fields of a case of logits: R rows of V logits of `type`, S sequences that
# hold up to L tokens (`own_rows`: row r is sequence r, else neighbouring rows
# share a sequence), n_bias biases a sequence, `mask`: some rows are under a
# grammar, `scale`: a temperature per sequence, `pen`: all penalties, or the
# repetition's only.


def listed():
    return [
        # one token of one sequence through a projection: latency counts
        dict(name="linear_t1", op="linear", T=1, K=2816, N=4096, g=128, tiled=True, xtype="f16", type="f16"),
        # a ragged small layer, odd channels, weights as the packer leaves them
        dict(name="linear_t3_ragged", op="linear", T=3, K=704, N=2111, g=64, tiled=False, xtype="bf16",
             type="bf16"),
        # sixteen sequences through a wide projection
        dict(name="linear_t16", op="linear", T=16, K=4096, N=11264, g=128, tiled=True, xtype="f16", type="f16"),
        # five sequences through the LM head, fp32 logits for the sampler
        dict(name="linear_t5_lmhead", op="linear", T=5, K=2816, N=262144, g=128, tiled=True, xtype="bf16",
             type="f32"),
        # the largest batch of the few-token form, untiled weights in groups of 64
        dict(name="linear_t64", op="linear", T=64, K=2816, N=16384, g=64, tiled=False, xtype="f16", type="f16"),
        # one short conversation, repetition penalty only: latency counts
        dict(name="adjust_one", op="adjust", R=1, V=32000, type="f32", S=1, L=300, own_rows=True, pen="rep",
             n_bias=0, mask=False, scale=False),
        # a batch of requests with every rule, an odd vocabulary
        dict(name="adjust_batch", op="adjust", R=48, V=100003, type="bf16", S=48, L=6000, own_rows=True,
             pen="all", n_bias=40, mask=True, scale=True),
        # a canvas of 256 positions of one sequence
        dict(name="adjust_canvas", op="adjust", R=256, V=262144, type="f32", S=1, L=4000, own_rows=False,
             pen="all", n_bias=0, mask=False, scale=False),
        # one sequence drawn with penalties over a long conversation
        dict(name="sample_one", op="sample", R=1, V=262144, type="f32", S=1, L=9000, own_rows=True, pen="all",
             n_bias=8, mask=False, scale=True, draw=True),
        # a batch of requests with every rule, drawn
        dict(name="sample_batch", op="sample", R=48, V=100003, type="bf16", S=48, L=6000, own_rows=True,
             pen="all", n_bias=40, mask=True, scale=True, draw=True),
        # a batch of long contexts, drawn, no grammar
        dict(name="sample_long", op="sample", R=64, V=262144, type="f32", S=64, L=60000, own_rows=True,
             pen="all", n_bias=0, mask=False, scale=True, draw=True),
        # a canvas of four sequences' drafts: confidences and the greedy tokens
        dict(name="sample_canvas", op="sample", R=256, V=262144, type="f32", S=4, L=8000, own_rows=False,
             pen="all", n_bias=0, mask=True, scale=False, draw=False),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["linear", "adjust", "sample"])
    if op == "linear":
        tiled = rng.random() < 0.6
        g = rng.choice([64, 128])
        while True:
            T = _log(rng, 1, 64)
            K = g * _log(rng, 1, 16384 // g)
            N = _log(rng, 16, 262144)
            if K * N <= MAX_WEIGHT // 2 and T * K * N <= 64 * MAX_WEIGHT // 8:
                break
        if tiled:
            N = (N + 15) // 16 * 16
        return dict(op=op, T=T, K=K, N=N, g=g, tiled=tiled, xtype=rng.choice(["f16", "bf16"]),
                    type=rng.choice(list(TYPES)))
    while True:
        R, V, L = _log(rng, 1, 256), _log(rng, 1000, 262144), _log(rng, 1, 60000)
        own_rows = rng.random() < 0.5
        S = R if own_rows else _log(rng, 1, R)
        if R * V <= MAX_LOGITS // 4 and S * L <= 64 * 60000:
            break
    case = dict(op=op, R=R, V=V, type=rng.choice(list(TYPES)), S=S, L=L, own_rows=own_rows,
                pen=rng.choice(["all", "all", "rep"]), n_bias=rng.choice([0, _log(rng, 1, 300)]),
                mask=rng.random() < 0.5, scale=rng.random() < 0.5)
    if op == "sample":
        case["draw"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & (2 ** 62 - 1))
    return g


def _pack4(g, N, K, group):
    """Weights N(0, 0.02), min/max rounded to 4 bits per group: q uint8
    [N, K/2], s and z fp16 [N, K/group]."""
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.empty((N, K // group), dtype=torch.float16, device=DEV)
    z = torch.empty_like(s)
    step = max(1, (1 << 26) // K)
    for n0 in range(0, N, step):
        n1 = min(N, n0 + step)
        w = torch.randn((n1 - n0, K // group, group), generator=g, device=DEV).mul_(0.02)
        lo, hi = w.amin(-1), w.amax(-1)
        sc = ((hi - lo) / 15).to(torch.float16)
        zp = torch.round(-lo / sc.float())
        codes = torch.round(w / sc.float()[..., None]).add_(zp[..., None]).clamp_(0, 15)
        codes = codes.to(torch.uint8).view(n1 - n0, K // 2, 2)
        q[n0:n1] = codes[..., 0] | (codes[..., 1] << 4)
        s[n0:n1] = sc
        z[n0:n1] = zp.to(torch.float16)
    return q, s, z


def _tokens(g, S, L, V):
    """Token sequences as text has them (few tokens many times, rank r about
    1/r of the time), the frequent ones spread over the vocabulary."""
    u = torch.rand((S, L), generator=g, device=DEV, dtype=torch.float64)
    rank = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
    return (rank * 7919 % V).to(torch.int32)


def _rules(g, case):
    S, R, V, L = case["S"], case["R"], case["V"], case["L"]
    uni = lambda lo, hi: lo + (hi - lo) * torch.rand(S, generator=g, device=DEV)
    r = dict(tokens=_tokens(g, S, L, V))
    r["lengths"] = (L * torch.rand(S, generator=g, device=DEV) * 1.25).clamp_(max=L).to(torch.int32)
    r["lengths"][0] = L
    if S > 2:
        r["lengths"][1] = 0                            # a sequence that has just begun
    r["prompt_lengths"] = (r["lengths"] * uni(0.1, 0.9)).to(torch.int32)
    r["repetition"] = uni(1.0, 1.4)
    if case["pen"] == "all":
        r["frequency"] = uni(0.0, 0.6)
        r["presence"] = uni(0.0, 0.8)
    if case["n_bias"]:
        n = min(case["n_bias"], V)
        ids = torch.rand((S, V), generator=g, device=DEV).topk(n, dim=1).indices if S * V <= 1 << 25 else \
            torch.stack([torch.randperm(V, generator=g, device=DEV)[:n] for _ in range(S)])
        r["bias_ids"] = ids.to(torch.int32)
        r["bias_ids"][torch.rand((S, n), generator=g, device=DEV) < 0.2] = -1     # unused places
        r["bias"] = 4.0 * torch.randn((S, n), generator=g, device=DEV)
    if case["scale"]:
        r["scale"] = 1.0 / uni(0.5, 1.5)
    if not case["own_rows"]:
        r["row_seq"] = (torch.arange(R, device=DEV) * S // R).to(torch.int32)
    if case["mask"]:
        # every other row is under a grammar, one leaves nearly everything,
        # another few tokens; with many rows one has come to a dead end
        M, W = (R + 1) // 2, (V + 31) // 32
        keep = torch.rand((M, 1), generator=g, device=DEV) < 0.5
        bits = torch.randint(0, 2 ** 31, (2, M, W), generator=g, device=DEV, dtype=torch.int32)
        sign = torch.randint(0, 2, (2, M, W), generator=g, device=DEV, dtype=torch.int32) << 31
        a, b = (bits | sign).unbind(0)
        wide = (torch.rand((M, W), generator=g, device=DEV) < 0.9).to(torch.int32) * -1
        few = (torch.rand((M, W), generator=g, device=DEV) < 0.02).to(torch.int32) * (a & b)
        mask = torch.where(keep, wide | a, few)
        if M > 8:
            mask[3] = 0
        r["mask"] = mask
        at = torch.arange(R, device=DEV, dtype=torch.int32)
        r["mask_row"] = torch.where(at % 2 == 0, at // 2, torch.full_like(at, -1))
    return r


def _inputs(case, seed):
    g = _gen(seed)
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        w = _pack4(g, N, K, case["g"])
        loud = torch.exp(0.5 * torch.randn(K, generator=g, device=DEV))    # some channels are louder
        x = (torch.randn((T, K), generator=g, device=DEV) * loud).to(TYPES[case["xtype"]])
        return dict(x=x, w=w)
    R, V = case["R"], case["V"]
    logits = torch.empty((R, V), dtype=TYPES[case["type"]], device=DEV)
    for r0 in range(0, R, 32):
        r1 = min(R, r0 + 32)
        logits[r0:r1] = 2.5 * torch.randn((r1 - r0, V), generator=g, device=DEV)
    # some tokens stand out, most of them tokens that the text has already
    rules = _rules(g, case)
    seq = rules["row_seq"].long() if "row_seq" in rules else torch.arange(R, device=DEV)
    at = torch.randint(0, case["L"], (R, 4), generator=g, device=DEV)
    top = torch.gather(rules["tokens"][seq].long(), 1, at)
    top[:, 3] = torch.randint(0, V, (R,), generator=g, device=DEV)
    high = 11.0 + 2.0 * torch.randn((R, 4), generator=g, device=DEV)
    logits.scatter_(1, top[:, :1], high[:, :1].to(logits.dtype))
    for k in range(1, 4):
        logits.scatter_(1, top[:, k:k + 1], high[:, k:k + 1].to(logits.dtype))
    return dict(logits=logits, rules=rules, seed=int(seed) * 2654435761 % 2 ** 64)


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        import w4a16_grouped_moe_amd as dg
        if case["op"] == "linear":
            w = (*st.pop("w"), case["g"])
            st["w"] = dg.pack_tiled(w) if case["tiled"] else w     # laid out once, when the weights are loaded
        else:
            st["rules"] = dg.LogitRules(**st["rules"])             # one per batch: a step changes its tensors
            if case["op"] == "sample":
                n = dg.sample_adjusted_workspace_bytes(case["R"], case["V"])
                st["ws_buf"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------- plain form

def _linear_plain(st):
    case = st["case"]
    q, s, z = st["w"]
    T, K, N, g = case["T"], case["K"], case["N"], case["g"]
    y = torch.empty((T, N), dtype=TYPES[case["type"]], device=q.device)
    x = st["x"].float()
    step = max(1, (1 << 27) // K)
    for n0 in range(0, N, step):
        n1 = min(N, n0 + step)
        codes = torch.stack((q[n0:n1] & 15, q[n0:n1] >> 4), dim=-1).view(n1 - n0, K // g, g).float()
        w = ((codes - z[n0:n1].float()[..., None]) * s[n0:n1].float()[..., None]).view(n1 - n0, K)
        y[:, n0:n1] = torch.matmul(x, w.t()).to(y.dtype)
    return y


def _history(r, S, V):
    """seen bool [S, V] and the count among the generated tokens fp32 [S, V]."""
    tok, n, p = r["tokens"], r["lengths"], r["prompt_lengths"]
    pos = torch.arange(tok.shape[1], device=tok.device)[None]
    live = (pos < n[:, None]) & (tok >= 0) & (tok < V)
    # what is not counted goes to a column of its own behind the last
    at = torch.where(live, tok, torch.full_like(tok, V)).long()
    seen = torch.zeros((S, V + 1), dtype=torch.bool, device=tok.device)
    seen.scatter_(1, at, True)
    at = torch.where(live & (pos >= p[:, None]), tok, torch.full_like(tok, V)).long()
    count = torch.zeros((S, V + 1), dtype=torch.float32, device=tok.device)
    count.scatter_add_(1, at, torch.ones_like(at, dtype=torch.float32))
    return seen[:, :V], count[:, :V]


def _blocks(st):
    """The adjusted logits, fp32, a block of rows at a time."""
    case, r = st["case"], st["rules"]
    R, V, S = case["R"], case["V"], case["S"]
    logits = st["logits"]
    dev = logits.device
    seen, count = _history(r, S, V)
    bias = None
    if "bias" in r:
        bias = torch.zeros((S, V + 1), dtype=torch.float32, device=dev)
        at = torch.where(r["bias_ids"] >= 0, r["bias_ids"], torch.full_like(r["bias_ids"], V)).long()
        bias.scatter_(1, at, r["bias"])
        bias = bias[:, :V]
    seq = r["row_seq"].long() if "row_seq" in r else torch.arange(R, device=dev)
    v = torch.arange(V, device=dev)
    step = max(1, (1 << 24) // V)
    for r0 in range(0, R, step):
        s = seq[r0:r0 + step]
        l = logits[r0:r0 + step].float()
        rep = r["repetition"][s][:, None]
        l = torch.where(seen[s], torch.where(l > 0, l / rep, l * rep), l)
        if "frequency" in r:
            c = count[s]
            l = torch.where(c > 0, l - r["frequency"][s][:, None] * c - r["presence"][s][:, None], l)
        if bias is not None:
            l = l + bias[s]
        if "scale" in r:
            l = l * r["scale"][s][:, None]
        if "mask" in r:
            m = r["mask_row"][r0:r0 + step].long()
            bits = (r["mask"][m.clamp(min=0)][:, v // 32] >> (v % 32).to(torch.int32)) & 1
            l = torch.where((bits != 0) | (m < 0)[:, None], l, torch.full_like(l, -math.inf))
        yield r0, l


def _philox(rows, blocks, seed):
    """Words [rows, blocks, 4] of Philox4x32-10 with counter {block, row, 0, 0}
    in 64-bit integers."""
    low = 0xFFFFFFFF

    def wide(m, a):
        # m * a, both below 2^32, as high and low words: halves of a at a time
        p0, p1 = m * (a & 0xFFFF), m * (a >> 16)
        t = (p0 >> 16) + (p1 & low)
        return (p1 >> 32 << 16) + (t >> 16), ((t & 0xFFFF) << 16) | (p0 & 0xFFFF)

    z = torch.zeros((rows.shape[0], blocks.shape[0]), dtype=torch.int64, device=rows.device)
    c0, c1, c2, c3 = z + blocks[None], z + rows[:, None], z, z
    k0, k1 = seed & low, seed >> 32
    for i in range(10):
        h0, l0 = wide(0xD2511F53, c0)
        h1, l1 = wide(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((c0, c1, c2, c3), dim=-1)


def _first_max(l):
    """The first place of a row's largest value; -1 where it holds nothing."""
    top = l.amax(1, keepdim=True)
    at = torch.arange(l.shape[1], device=l.device)[None]
    first = torch.where(l == top, at, torch.full_like(at, l.shape[1])).amin(1)
    return torch.where(top[:, 0] == -math.inf, torch.full_like(first, -1), first).to(torch.int32)


def _sample_plain(st):
    case = st["case"]
    R, V = case["R"], case["V"]
    dev = st["logits"].device
    entropy = torch.empty(R, dtype=torch.float32, device=dev)
    argmax = torch.empty(R, dtype=torch.int32, device=dev)
    sample = torch.empty(R, dtype=torch.int32, device=dev) if case["draw"] else None
    for r0, l in _blocks(st):
        r1 = r0 + l.shape[0]
        top = l.amax(1, keepdim=True)
        none = top == -math.inf
        d = l - torch.where(none, torch.zeros_like(top), top)
        e = torch.exp(d)
        z = e.sum(1)
        s = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1)
        h = torch.log(z) - s / z
        entropy[r0:r1] = torch.where(none[:, 0], torch.zeros_like(h), h)
        argmax[r0:r1] = _first_max(l)
        if sample is not None:
            # the noise in 64 bits: a row's two best scores may lie close together
            blocks = torch.arange((V + 3) // 4, device=dev)
            w = _philox(torch.arange(r0, r1, device=dev), blocks, st["seed"]).view(r1 - r0, -1)[:, :V]
            u = ((w >> 9).double() + 0.5) * 2.0 ** -23
            sample[r0:r1] = _first_max(l.double() - torch.log(-torch.log(u)))
    return entropy, sample, argmax


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import w4a16_grouped_moe_amd as dg
        if op == "linear":
            return dg.w4a16_linear_few(state["x"], state["w"], dtype=TYPES[case["type"]])
        if op == "adjust":
            return dg.adjust_logits(state["logits"], state["rules"])
        out = dg.sample_adjusted(state["logits"], state["rules"], state["seed"], draw=case["draw"],
                                 workspace=state["ws_buf"])
        return out if case["draw"] else (out[0], out[2])
    if op == "linear":
        return _linear_plain(state)
    if op == "adjust":
        out = torch.empty(state["logits"].shape, dtype=torch.float32, device=state["logits"].device)
        for r0, l in _blocks(state):
            out[r0:r0 + l.shape[0]] = l
        return out
    entropy, sample, argmax = _sample_plain(state)
    return (entropy, sample, argmax) if case["draw"] else (entropy, argmax)


def work(case):
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": N * K // 2 + N * (K // case["g"]) * 4 + T * K * 2 + T * N * BYTES[case["type"]],
                "flops": 2.0 * T * N * K}
    R, V, S, L = case["R"], case["V"], case["S"], case["L"]
    n = R * V
    # lengths are 5/8 of L on average, 0.6 L with the longest cut off at L
    rules = S * (0.6 * L * 4 + case["n_bias"] * 8 + 32)
    rules += ((R + 1) // 2) * ((V + 31) // 32) * 4 if case["mask"] else 0
    if case["op"] == "adjust":
        return {"bytes": n * (BYTES[case["type"]] + 4) + rules, "flops": 1.0 * n}
    return {"bytes": n * BYTES[case["type"]] + rules + 12 * R, "flops": (60.0 if case["draw"] else 8.0) * n}


# ---------------------------------------------------------------- definitions in 64 bits

def _exact_linear(case, st):
    q, s, z = st["w"]
    g, N = case["g"], case["N"]
    x = st["x"].double()
    y = torch.empty((case["T"], N), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 26) // case["K"])
    for n0 in range(0, N, step):
        sl = slice(n0, min(N, n0 + step))
        w = torch.empty((sl.stop - n0, case["K"]), dtype=torch.float64, device=DEV)
        w[:, 0::2] = q[sl].bitwise_and(15).double()
        w[:, 1::2] = q[sl].bitwise_right_shift(4).double()
        w -= z[sl].double().repeat_interleave(g, 1)
        w *= s[sl].double().repeat_interleave(g, 1)
        y[:, sl] = x @ w.T
    return y


def _exact_row(case, st, host, r):
    """One row's adjusted logits in 64 bits: token by token rules, applied to
    the tokens that have any."""
    rules = st["rules"]
    V = case["V"]
    s = int(host["row_seq"][r]) if "row_seq" in host else r
    l = st["logits"][r].double()
    n, p = int(host["lengths"][s]), int(host["prompt_lengths"][s])
    every = torch.unique(rules["tokens"][s, :n].long())
    rep = host["repetition"][s].item()
    v = l[every]
    l[every] = torch.where(v > 0, v / rep, v * rep)
    if "frequency" in host:
        made, times = torch.unique(rules["tokens"][s, p:n].long(), return_counts=True)
        l[made] -= host["frequency"][s].item() * times.double() + host["presence"][s].item()
    if "bias" in host:
        ids = rules["bias_ids"][s].long()
        l[ids[ids >= 0]] += rules["bias"][s][ids >= 0].double()
    if "scale" in host:
        l = l * host["scale"][s].item()
    if "mask" in host:
        m = int(host["mask_row"][r])
        if m >= 0:
            words = rules["mask"][m].long()
            allowed = torch.bitwise_and(words[:, None] >> torch.arange(32, device=DEV), 1).view(-1)[:V] == 1
            l = l.masked_fill(~allowed, -math.inf)
    return l


def _exact_score(l, r, seed):
    """l + G of one row, in 64 bits."""
    M = 2 ** 32
    c = [torch.arange((l.shape[0] + 3) // 4, device=DEV), r, 0, 0]
    key = [seed % M, seed // M]

    def product(a, b):
        """High and low words of a * b for b below 2^32 (a tensor or a number)."""
        if not torch.is_tensor(b):
            return a * b // M, a * b % M
        lo, hi = b % 65536 * a, b // 65536 * a
        total = hi % 65536 * 65536 + lo % M
        return hi // 65536 + lo // M + total // M, total % M

    for i in range(10):
        h0, l0 = product(0xD2511F53, c[0])
        h1, l1 = product(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % M, (key[1] + 0xBB67AE85) % M]
    w = torch.stack(torch.broadcast_tensors(*c), dim=1).reshape(-1)[:l.shape[0]]
    u = (torch.div(w, 512, rounding_mode="floor").double() + 0.5) / 2 ** 23
    return l - torch.log(-torch.log(u))


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "linear":
        return _exact_linear(case, st)
    host = {k: v.cpu() for k, v in st["rules"].items() if k not in ("tokens", "mask")}
    host["mask"] = None
    host = {k: v for k, v in host.items() if k in st["rules"]}
    R = case["R"]
    if case["op"] == "adjust":
        out = torch.empty(st["logits"].shape, dtype=torch.float64, device=DEV)
        for r in range(R):
            out[r] = _exact_row(case, st, host, r)
        return out
    entropy = torch.zeros(R, dtype=torch.float64, device=DEV)
    argmax = torch.full((R,), -1, dtype=torch.int32, device=DEV)
    sample = torch.full((R,), -1, dtype=torch.int32, device=DEV)
    for r in range(R):
        l = _exact_row(case, st, host, r)
        live = torch.nonzero(l > -math.inf)[:, 0]
        if live.numel() == 0:
            continue
        v = l[live]
        logp = v - torch.logsumexp(v, 0)
        entropy[r] = -(logp.exp() * logp).sum()
        argmax[r] = live[torch.nonzero(v == v.max())[0, 0]]
        if case["draw"]:
            score = _exact_score(l, r, st["seed"])[live]
            sample[r] = live[torch.nonzero(score == score.max())[0, 0]]
    return (entropy, sample, argmax) if case["draw"] else (entropy, argmax)
