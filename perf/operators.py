"""The operators of a serving step at few tokens, as measured cases.

A step of a small batch runs the routed experts for a few tokens, and its
dense products (projections, the LM head) on 8-bit integers with one scale
per token and one per output channel:

* ``moe``     the whole routed-expert layer (W4A16 experts) for a few tokens,
              from the router's ids and weights or from its logits;
* ``rows``    symmetric 8-bit quantisation of rows (a token's activations, a
              channel's weights), one fp32 scale per row;
* ``linear``  the product of 8-bit rows with 8-bit channels and their scales;
* ``tokens``  the same product from fp16 / bf16 / fp32 activations, quantised
              per token on the way.

``own`` false: plain elementary torch operations in 32 bits. ``own`` true:
the calls a user makes of ``w4a16_grouped_moe_amd``. ``exact`` computes the
definitions in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}

# The layer's widths (d, m), experts and choices per token are this
# repository's; a dense layer's K is the layer's d.
LAYER = {"E": 128, "topk": 8, "d": 2816, "m": 704, "gu_g": 128, "dn_g": 64, "tiled": True}

# The largest work of a listed case, which drawn ones stay below.
MAX_MACS = 256 * 262144 * 2816
MAX_WEIGHT = 262144 * 2816


def listed():
    return [
        # one token of one sequence, straight from the router's logits: the
        # shortest step there is, where launches and latency count
        dict(LAYER, name="moe_t1_routed", op="moe", T=1, routed=True, zipf=0.0, pad=0),
        # a handful of sequences, ids at hand, two rows of the batch being
        # padding (their ids are -1 and their outputs zero)
        dict(LAYER, name="moe_t6_padded", op="moe", T=6, routed=False, zipf=0.0, pad=2),
        # sixteen tokens whose router prefers some experts
        dict(LAYER, name="moe_t16_skew", op="moe", T=16, routed=True, zipf=1.2, pad=0),
        # the largest batch of the few-token form: nearly every expert is read
        dict(LAYER, name="moe_t64", op="moe", T=64, routed=False, zipf=0.0, pad=0),
        # a canvas of activations before a dense layer
        dict(name="rows_canvas", op="rows", rows=256, K=2816, type="f16", skip=0),
        # a prompt's activations, a slice of a wider tensor (strided rows, an
        # odd length)
        dict(name="rows_prompt", op="rows", rows=16001, K=2803, type="bf16", skip=45),
        # a canvas through a projection
        dict(name="linear_canvas", op="linear", T=256, K=2816, N=4096, type="f16"),
        # a ragged batch through a small layer, odd channels
        dict(name="linear_ragged", op="linear", T=77, K=704, N=2111, type="bf16"),
        # a prompt through a wide projection: the matrix rate counts
        dict(name="linear_prompt", op="linear", T=4096, K=2816, N=11264, type="bf16"),
        # a canvas through the LM head, fp32 logits for the sampler
        dict(name="linear_lmhead", op="linear", T=256, K=2816, N=262144, type="f32"),
        # one token through a projection, from its activations
        dict(name="tokens_t1", op="tokens", T=1, K=2816, N=4096, xtype="f16", type="f16"),
        # five tokens through the LM head, from their activations
        dict(name="tokens_lmhead", op="tokens", T=5, K=2816, N=262144, xtype="bf16", type="f32"),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["moe", "rows", "linear", "tokens"])
    if op == "moe":
        while True:
            gu_g, dn_g = rng.choice([(128, 64), (128, 128), (64, 64), (64, 128)])
            E = _log(rng, 4, 256)
            topk = rng.randint(1, min(8, E))
            T = _log(rng, 1, 64)
            d = gu_g * _log(rng, 256 // gu_g, 4096 // gu_g)
            m = dn_g * _log(rng, 128 // dn_g, 1408 // dn_g)
            if E * 3 * m * d <= MAX_WEIGHT:
                break
        return dict(op="moe", E=E, topk=topk, T=T, d=d, m=m, gu_g=gu_g, dn_g=dn_g,
                    tiled=rng.random() < 0.7, routed=rng.random() < 0.5,
                    zipf=rng.choice([0.0, 0.0, 1.2]), pad=rng.randint(0, T // 2))
    if op == "rows":
        while True:
            rows, K = _log(rng, 1, 65536), _log(rng, 16, 16384)
            if rows * K <= 16001 * 2803:
                break
        return dict(op="rows", rows=rows, K=K, type=rng.choice(list(TYPES)),
                    skip=rng.choice([0, 0, rng.randint(1, 64)]))
    while True:
        T = _log(rng, 1, 4096) if op == "linear" else _log(rng, 1, 512)
        K = _log(rng, 64, 16384)
        N = _log(rng, 16, 262144)
        if T * K * N <= MAX_MACS // 2 and K * N <= MAX_WEIGHT // 2 and T * N <= 256 * 262144:
            break
    case = dict(op=op, T=T, K=K, N=N, type=rng.choice(list(TYPES)))
    if op == "linear":
        case["K"] = (K + 15) // 16 * 16           # rows of 8-bit values come in whole 16 bytes
    else:
        case["xtype"] = rng.choice(list(TYPES))
    return case


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & (2 ** 62 - 1))
    return g


def _pack4(g, E, N, K, group):
    """Weights N(0, 0.02), min/max rounded to 4 bits per group: q uint8
    [E, N, K/2], s and z fp16 [E, N, K/group]."""
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.empty((E, N, K // group), dtype=torch.float16, device=DEV)
    z = torch.empty_like(s)
    for e0 in range(0, E, 16):
        e1 = min(E, e0 + 16)
        w = torch.randn((e1 - e0, N, K // group, group), generator=g, device=DEV).mul_(0.02)
        lo, hi = w.amin(-1), w.amax(-1)
        sc = ((hi - lo) / 15).to(torch.float16)
        zp = torch.round(-lo / sc.float())
        codes = torch.round(w / sc.float()[..., None]).add_(zp[..., None]).clamp_(0, 15)
        codes = codes.to(torch.uint8).view(e1 - e0, N, K // 2, 2)
        q[e0:e1] = codes[..., 0] | (codes[..., 1] << 4)
        s[e0:e1] = sc
        z[e0:e1] = zp.to(torch.float16)
    return q, s, z


def _activations(g, rows, cols, dtype):
    """N(0, 1) with some channels several times louder, as hidden states have."""
    loud = torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV))
    return (torch.randn((rows, cols), generator=g, device=DEV) * loud).to(dtype)


def _int8_rows(g, rows, cols):
    """8-bit codes of normally distributed rows and their scales."""
    q = torch.empty((rows, cols), dtype=torch.int8, device=DEV)
    for r0 in range(0, rows, 65536):
        r1 = min(rows, r0 + 65536)
        q[r0:r1] = torch.randn((r1 - r0, cols), generator=g, device=DEV).mul_(33.0).round_().clamp_(-127, 127)
    s = (0.02 / 33.0) * torch.exp(0.2 * torch.randn(rows, generator=g, device=DEV))
    return q, s


def _up16(k):
    return (k + 15) // 16 * 16


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "moe":
        T, E, d, m = case["T"], case["E"], case["d"], case["m"]
        st = dict(gu=_pack4(g, E, 2 * m, d, case["gu_g"]), dn=_pack4(g, E, d, m, case["dn_g"]))
        st["x"] = torch.randn((T, d), generator=g, device=DEV).to(torch.float16)
        logits = torch.randn((T, E), generator=g, device=DEV)
        if case["zipf"]:
            rank = torch.randperm(E, generator=g, device=DEV).float() + 1
            logits = logits - case["zipf"] * torch.log(rank)
        st["logits"] = logits
        if not case["routed"]:
            ids, w = _route(logits, case["topk"])
            if case["pad"]:
                ids[T - case["pad"]:] = -1
            st["ids"], st["w"] = ids, w
        return st
    if op == "rows":
        wide = _activations(g, case["rows"], case["K"] + case["skip"], TYPES[case["type"]])
        return dict(x=wide[:, :case["K"]])
    T, K, N = case["T"], case["K"], case["N"]
    st = {}
    st["wq"], st["ws"] = _int8_rows(g, N, _up16(K))
    if op == "linear":
        st["xq"], st["xs"] = _int8_rows(g, T, K)
    else:
        st["x"] = _activations(g, T, K, TYPES[case["xtype"]])
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        import w4a16_grouped_moe_amd as dg
        op = case["op"]
        if op == "moe":
            gu, dn = (*st.pop("gu"), case["gu_g"]), (*st.pop("dn"), case["dn_g"])
            if case["tiled"]:                     # laid out once, when the weights are loaded
                gu, dn = dg.pack_tiled(gu), dg.pack_tiled(dn)
            st["gu"], st["dn"] = gu, dn
            n = dg.moe_few_workspace_bytes(case["T"], case["topk"], case["E"], case["d"],
                                           case["m"], gu[3], dn[3])
            st["ws_buf"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
        elif op == "tokens":
            n = dg.w8a8_workspace_bytes(case["T"], case["K"])
            st["ws_buf"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------- plain form

def _route(logits, topk):
    """The topk largest logits of each token (equal ones by the lower id) and
    the softmax over them."""
    v, i = torch.sort(logits, dim=1, descending=True, stable=True)
    v, i = v[:, :topk], i[:, :topk]
    p = torch.exp(v - v[:, :1])
    return i.to(torch.int32), p / p.sum(1, keepdim=True)


def _deq(q, s, z):
    """(code - zero) * scale of packed weights [..., N, K/2] in fp32."""
    n, k = q.shape[-2], q.shape[-1] * 2
    codes = torch.stack((q & 15, q >> 4), dim=-1).view(*q.shape[:-1], k)
    grouped = codes.view(*q.shape[:-1], s.shape[-1], k // s.shape[-1]).float()
    return ((grouped - z.float()[..., None]) * s.float()[..., None]).view(*q.shape[:-2], n, k)


def _gelu(v):
    return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))


def _moe_plain(st):
    case = st["case"]
    m, E, T, topk = case["m"], case["E"], case["T"], case["topk"]
    x = st["x"].float()
    ids, w = _route(st["logits"], topk) if case["routed"] else (st["ids"], st["w"])
    live = (ids >= 0) & (ids < E)
    out = torch.zeros((T, case["d"]), dtype=torch.float32, device=x.device)
    if 2 * T < E:
        # each token's experts gathered, where that is less than all experts
        at = ids.clamp(0, E - 1).long()
        wt = torch.where(live, w, torch.zeros_like(w))
        for t in range(T):
            wgu = _deq(*(p[at[t]] for p in st["gu"]))
            a = torch.matmul(wgu, x[t])
            h = _gelu(a[:, :m]) * a[:, m:]
            wdn = _deq(*(p[at[t]] for p in st["dn"]))
            y = torch.matmul(wdn, h[..., None])[..., 0]
            out[t] = (wt[t][:, None] * y).sum(0)
    else:
        for e in range(E):
            a = torch.matmul(x, _deq(*(p[e] for p in st["gu"])).t())
            h = _gelu(a[:, :m]) * a[:, m:]
            y = torch.matmul(h, _deq(*(p[e] for p in st["dn"])).t())
            we = torch.where(ids == e, w, torch.zeros_like(w)).sum(1)
            out += we[:, None] * y
    return out.to(torch.float16)


def _quant_plain(x):
    xf = x.float()
    amax = xf.abs().amax(1)
    s = amax / torch.full_like(amax, 127.0)
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = torch.round(xf / s[:, None]).clamp(-127, 127)
    return q, s


def _product_plain(xq, xs, wq, ws, dtype):
    """The codes' sums are whole numbers below 2^24 for these inputs, which
    32 bits hold exactly."""
    T, N = xq.shape[0], wq.shape[0]
    y = torch.empty((T, N), dtype=dtype, device=xq.device)
    xf = xq.float()
    for n0 in range(0, N, 32768):
        n1 = min(N, n0 + 32768)
        acc = torch.matmul(xf, wq[n0:n1, :xf.shape[1]].float().t())
        y[:, n0:n1] = (acc * xs[:, None] * ws[None, n0:n1]).to(dtype)
    return y


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import w4a16_grouped_moe_amd as dg
        if op == "moe":
            if case["routed"]:
                return dg.moe_few_routed(state["x"], state["logits"], case["topk"], state["gu"],
                                         state["dn"], workspace=state["ws_buf"])
            return dg.moe_few(state["x"], state["ids"], state["w"], state["gu"], state["dn"],
                              workspace=state["ws_buf"])
        if op == "rows":
            return dg.quantize_rows_i8(state["x"])
        if op == "linear":
            return dg.w8a8_linear(state["xq"], state["xs"], (state["wq"], state["ws"]),
                                  dtype=TYPES[case["type"]])
        return dg.w8a8_linear_tokens(state["x"], (state["wq"], state["ws"]),
                                     dtype=TYPES[case["type"]], workspace=state["ws_buf"])
    if op == "moe":
        return _moe_plain(state)
    if op == "rows":
        q, s = _quant_plain(state["x"])
        pad = _up16(case["K"]) - case["K"]
        return torch.nn.functional.pad(q.to(torch.int8), (0, pad)), s
    dtype = TYPES[case["type"]]
    if op == "linear":
        return _product_plain(state["xq"], state["xs"], state["wq"], state["ws"], dtype)
    q, s = _quant_plain(state["x"])
    return _product_plain(q, s, state["wq"], state["ws"], dtype)


def _experts_read(case):
    """The number of different experts that the tokens choose, on average
    (a few simulated routings)."""
    rng = np.random.default_rng(5)
    T, E, k = case["T"] - (0 if case["routed"] else case["pad"]), case["E"], case["topk"]
    n = 0
    for _ in range(8):
        lg = rng.standard_normal((T, E))
        if case["zipf"]:
            lg -= case["zipf"] * np.log(np.arange(1, E + 1))
        n += len(np.unique(np.argpartition(-lg, k - 1, axis=1)[:, :k]))
    return n / 8


def work(case):
    op = case["op"]
    if op == "moe":
        T, d, m, k = case["T"], case["d"], case["m"], case["topk"]
        per_expert = (3 * m * d // 2 + 4 * (2 * m * d // case["gu_g"]) + 4 * (d * m // case["dn_g"]))
        live = T - (0 if case["routed"] else case["pad"])
        route = T * case["E"] * 4 if case["routed"] else T * k * 8
        return {"bytes": _experts_read(case) * per_expert + 4 * T * d + route,
                "flops": 2.0 * live * k * 3 * m * d}
    if op == "rows":
        n = case["rows"] * case["K"]
        return {"bytes": n * BYTES[case["type"]] + case["rows"] * (_up16(case["K"]) + 4),
                "flops": 3.0 * n}
    T, K, N = case["T"], case["K"], case["N"]
    x = T * (K + 4) if op == "linear" else T * K * BYTES[case["xtype"]]
    return {"bytes": x + N * (K + 4) + T * N * BYTES[case["type"]], "flops": 2.0 * T * N * K}


# ---------------------------------------------------------------- definitions in 64 bits

def _exact_moe(case, st):
    x = st["x"].double()
    T, E, m, topk = case["T"], case["E"], case["m"], case["topk"]
    if case["routed"]:
        lg = st["logits"].double().cpu().numpy()
        chosen = np.argsort(-lg, axis=1, kind="stable")[:, :topk]
        v = np.take_along_axis(lg, chosen, 1)
        p = np.exp(v - v.max(1, keepdims=True))
        weight = p / p.sum(1, keepdims=True)
    else:
        chosen = st["ids"].cpu().numpy()
        weight = st["w"].double().cpu().numpy()

    def matrix(pack, e):
        q, s, z = (p[e] for p in pack)
        q = q.to(torch.int64)
        codes = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=DEV)
        codes[:, 0::2] = q.bitwise_and(15)
        codes[:, 1::2] = q.bitwise_right_shift(4)
        rep = codes.shape[1] // s.shape[1]
        return (codes - z.double().repeat_interleave(rep, 1)) * s.double().repeat_interleave(rep, 1)

    out = torch.zeros((T, case["d"]), dtype=torch.float64, device=DEV)
    for e in sorted({int(i) for i in chosen.ravel() if 0 <= i < E}):
        rows, slots = np.nonzero(chosen == e)
        both = x[torch.as_tensor(rows, device=DEV)] @ matrix(st["gu"], e).T
        gate, up = both[:, :m], both[:, m:]
        inner = (2.0 / math.pi) ** 0.5 * gate * (1.0 + 0.044715 * gate ** 2)
        h = gate / (1.0 + torch.exp(-2.0 * inner)) * up
        y = h @ matrix(st["dn"], e).T
        out.index_add_(0, torch.as_tensor(rows, device=DEV),
                       torch.as_tensor(weight[rows, slots], device=DEV)[:, None] * y)
    return out


def _exact_quant(x):
    """Scale and codes with the definition's roundings to fp32 (the scale, the
    quotient): a quotient in 64 bits rounded to 32 is the correctly rounded
    one."""
    xd = x.double()
    top = torch.max(xd.abs(), dim=1).values
    s = (top / 127.0).float().double()
    s[s == 0] = 1.0
    ratio = (xd / s.unsqueeze(1)).float().double()
    return torch.round(ratio).clamp_(-127, 127), s


def _exact_product(xq, xs, wq, ws):
    T, K = xq.shape
    y = torch.empty((T, wq.shape[0]), dtype=torch.float64, device=DEV)
    for n0 in range(0, wq.shape[0], 16384):
        part = wq[n0:n0 + 16384, :K].double()
        y[:, n0:n0 + 16384] = (xq.double() @ part.T) * (xs.double()[:, None] * ws[n0:n0 + 16384].double())
    return y


def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op == "moe":
        return _exact_moe(case, st)
    if op == "rows":
        q, s = _exact_quant(st["x"])
        codes = torch.zeros((case["rows"], _up16(case["K"])), dtype=torch.float64, device=DEV)
        codes[:, :case["K"]] = q
        return codes, s
    if op == "linear":
        return _exact_product(st["xq"], st["xs"], st["wq"], st["ws"])
    q, s = _exact_quant(st["x"])
    return _exact_product(q, s, st["wq"], st["ws"])
