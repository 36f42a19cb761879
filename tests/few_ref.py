"""Plain 64-bit forms of the few-token operators and the error each kernel
output may have (test helper).

The bounds count the kernel's roundings, no measured slack: u32 = 2^-24 is
half a step of fp32, u16 = 2^-11 of fp16. A sum of n fp32 terms in any order
is off by at most n * u32 * (sum of the terms' magnitudes) (first order; the
factor 1.01 covers the higher ones for the n used here).
"""
from __future__ import annotations

import numpy as np
import torch

U32, U16 = 2.0 ** -24, 2.0 ** -11
FP16_TINY = 2.0 ** -25          # half a step of fp16's subnormals


def dequant(pack, e):
    """One expert's weights (q - z) * s, float64 [N, K], from the packed
    tensors (canonical layout, numpy)."""
    q, s, z, g = pack
    codes = np.stack((q[e] & 15, q[e] >> 4), axis=-1).reshape(q.shape[1], -1).astype(np.float64)
    rep = lambda v: np.repeat(v[e].astype(np.float64), g, axis=1)
    return codes, rep(s), rep(z)


def moe(x, ids, w, gu, dn, E):
    """out float64 [T, d] of the routed-expert layer and the bound on the
    kernel's error. x fp16, ids int, w fp32 (numpy), packs canonical numpy.

    The kernel: gate and up are fp32 sums over K of x * (q - z) (exact
    factors; products of an 11-bit and a 5- to 12-bit integer are exact in
    fp32), the group's scale applied in fp32 to each group's sum: at most
    K + 3 K / g + 16 roundings touch a term, and K + 64 covers them (a sum over
    a group, its product with s, the sum of groups and of eight waves). gelu
    in fp32: a hardware exp2 and reciprocal of about 1 ulp each and eight other
    roundings, the argument's relative error (8 u32) times |d log gelu / d log v|
    <= 1 + |2 u| with |2 u| <= 40 where the result matters: 512 u32. H is rounded
    to fp16 once, down is an fp32 sum as above, out is an fp32 sum over k
    rounded to fp16 once."""
    T, d = x.shape
    m = dn[0].shape[2] * 2
    out, bound = np.zeros((T, d)), np.zeros((T, d))
    xf = x.astype(np.float64)
    for e in sorted({int(i) for i in ids.ravel() if 0 <= i < E}):
        cg, sg, zg = dequant(gu, e)
        cd, sd, zd = dequant(dn, e)
        wg, wd = (cg - zg) * sg, (cd - zd) * sd
        t, k = np.nonzero(ids == e)
        both = xf[t] @ wg.T
        mag = np.abs(xf[t]) @ np.abs(wg).T
        gam = 1.01 * (d + 64) * U32
        gate, up = both[:, :m], both[:, m:]
        dgate, dup = gam * mag[:, :m], gam * mag[:, m:]
        act = 0.5 * gate * (1 + np.tanh(np.sqrt(2 / np.pi) * (gate + 0.044715 * gate ** 3)))
        h = act * up
        dact = 1.13 * dgate + 512 * U32 * np.abs(act) + 2.0 ** -120   # |gelu'| <= 1.13
        dh = dact * (np.abs(up) + dup) + np.abs(act) * dup + 2 * U32 * np.abs(h)
        dh = dh + U16 * (np.abs(h) + dh) + FP16_TINY
        y = h @ wd.T
        gam = 1.01 * (m + 64) * U32
        dy = dh @ np.abs(wd).T + gam * (np.abs(h) + dh) @ np.abs(wd).T
        wt = w[t, k].astype(np.float64)[:, None]
        np.add.at(out, t, wt * y)
        np.add.at(bound, t, np.abs(wt) * (dy + (ids.shape[1] + 2) * U32 * (np.abs(y) + dy)))
    return out, bound + U16 * (np.abs(out) + bound) + FP16_TINY


def quantize_rows(x):
    """(codes int8 [rows, K up to 16], scales fp32) by the definition, from a
    torch tensor on the CPU."""
    xf = x.float().numpy()
    rows, K = xf.shape
    with np.errstate(all="ignore"):
        top = np.abs(xf).max(axis=1)
        s = (top / np.float32(127)).astype(np.float32)
        s[s == 0] = 1
        q = np.clip(np.rint(xf / s[:, None]), -127, 127)
    bad = ~np.isfinite(top)
    s[bad], q[bad] = np.nan, 0
    codes = np.zeros((rows, (K + 15) // 16 * 16), dtype=np.int8)
    codes[:, :K] = q.astype(np.int8)
    return codes, s


def product(xq, xs, wq, ws, dtype):
    """The 8-bit product by its definition (exact 64-bit integer sums below
    2^53 taken through float64, then the stated fp32 roundings), as a torch
    tensor of ``dtype``."""
    acc = (xq.astype(np.float64) @ wq.astype(np.float64).T).astype(np.float32)
    with np.errstate(all="ignore"):
        y = (acc * xs[:, None]).astype(np.float32) * ws[None, :]
    return torch.from_numpy(y.astype(np.float32)).to(dtype)


def same_bits(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Equal bits, any NaN equal to any other."""
    a, b = a.cpu(), b.cpu()
    na, nb = torch.isnan(a), torch.isnan(b)
    it = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(na, nb) and torch.equal(a.view(it)[~na], b.view(it)[~nb])
